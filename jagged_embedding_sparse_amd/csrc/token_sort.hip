// The tokens of a batch sorted by row: the CSR that the gradient reads.
//
// A stable LSD radix sort of (row, token), so a row's tokens keep their order.
// Dropped tokens (padding, IDs outside the table) take the row number behind
// the last one, which sorts last and is left out of the result. At these sizes
// launches cost more than the data: the dedup's path for the same items takes
// eleven dependent launches (about 60 us up to 262144 tokens). Here
//  - up to kSmall tokens one workgroup sorts in LDS and writes the CSR;
//  - up to kMidTiles tiles a pass is two launches (digit counts per tile; a
//    scatter in which every workgroup sums the counts before it itself instead
//    of a scan between them), and the CSR is one more, whose workgroups count
//    the rows before their tile themselves, or read them from a second one
//    where there are many;
//  - larger batches go through the dedup with one shard, whose tiled scans
//    they need.
#include <algorithm>

#include "common.hpp"

namespace fs {
namespace {

constexpr int kThreads = 256;

// the sort key of token i: its row, or `rows` if it is dropped
__device__ __forceinline__ uint32_t token_key(int64_t id, int64_t rows, int64_t padding, bool& bad) {
  const bool out = id < 0 || id >= rows;
  bad |= out && id != padding;
  return out || id == padding ? (uint32_t)rows : (uint32_t)id;
}

struct SortOut {
  int64_t* unique;
  int64_t* unique_offsets;
  int32_t* seg;
  int32_t* bm;
  int32_t* uid;
  int64_t* counts;
};

__device__ __forceinline__ void write_totals(const SortOut& o, int64_t U, int32_t valid) {
  o.seg[U] = valid;
  o.unique_offsets[0] = 0;
  o.unique_offsets[1] = U;
  o.counts[0] = o.counts[2] = U;
  o.counts[1] = o.counts[3] = 0;
}

// ---------------------------------------------------------------- one pass
// Items of a workgroup: wave w holds items 256 w + 64 i + lane, i = 0..3, so
// that the waves' rounds follow the items' order.
constexpr int kRounds = 4;
constexpr int kWaveItems = kWave * kRounds;

// Stable places of a workgroup's items by a digit. place[i] = the item's place
// among the workgroup's items of the same digit, plus start(digit), which is
// called for each digit with the workgroup's count of it by the thread that
// owns the digit; it may use barriers, so all threads call it `per` times.
// `count` and `peers` are LDS of [waves][bins] each, peers all zero on entry
// and exit.
template <int NT, int BITS, typename Start>
__device__ __forceinline__ void digit_places(const uint32_t (&key)[kRounds], int32_t n, int shift,
                                             int bits, uint32_t (*count)[1 << BITS],
                                             uint64_t (*peers)[1 << BITS], Start start,
                                             uint32_t (&place)[kRounds]) {
  constexpr int kWaves = NT / kWave;
  const int w = threadIdx.x / kWave, l = lane(), bins = 1 << bits;
  const uint32_t mask = (uint32_t)bins - 1;
  const int32_t wn = n - w * kWaveItems;  // this wave's items
  for (int b = l; b < bins; b += kWave) count[w][b] = 0;
  // a wave's LDS operations complete in order
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    if (i * kWave + l < wn) atomicAdd(&count[w][(key[i] >> shift) & mask], 1u);
  __syncthreads();
  for (int b0 = 0; b0 < bins; b0 += NT) {  // uniform
    const int b = b0 + threadIdx.x;
    uint32_t tot = 0;
    if (b < bins) {
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        const uint32_t c = count[x][b];
        count[x][b] = tot;
        tot += c;
      }
    }
    const uint32_t at = start(b, tot);
    if (b < bins) {
#pragma unroll
      for (int x = 0; x < kWaves; ++x) count[x][b] += at;
    }
  }
  __syncthreads();
  const uint64_t lt = lanemask_lt();
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    if (i * kWave < wn) {  // uniform per wave
      const bool on = i * kWave + l < wn;
      const uint32_t d = on ? (key[i] >> shift) & mask : 0u;
      const uint64_t same = lds_peers(peers[w], d, on);
      const uint32_t at = count[w][d];
      if (on) {
        place[i] = at + (uint32_t)popc(same & lt);
        if ((same & lt) == 0) count[w][d] = at + (uint32_t)popc(same);
      }
    }
  }
}

// ---------------------------------------------------------------- small
constexpr int kSmallBits = 8;

template <int NT>
__global__ void __launch_bounds__(NT)
k_token_sort_small(const int64_t* __restrict__ ids, int32_t n, int64_t rows, int64_t padding,
                   int32_t kbits, SortOut o, int32_t* __restrict__ err) {
  constexpr int kItems = NT * kRounds;
  __shared__ uint32_t s_key[kItems];
  __shared__ int32_t s_val[kItems];
  __shared__ uint32_t count[NT / kWave][1 << kSmallBits];
  __shared__ uint64_t peers[NT / kWave][1 << kSmallBits];
  __shared__ uint32_t tmp[17];
  const int w = threadIdx.x / kWave, l = lane();
  uint32_t key[kRounds], place[kRounds];
  int32_t val[kRounds];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    val[i] = w * kWaveItems + i * kWave + l;
    key[i] = val[i] < n ? token_key(ids[val[i]], rows, padding, bad) : (uint32_t)rows;
  }
  flag_err(err, bad, FS_EF_ID_RANGE);
  for (int b = l; b < 1 << kSmallBits; b += kWave) peers[w][b] = 0;
  const int passes = (kbits + kSmallBits - 1) / kSmallBits;
  for (int p = 0, shift = 0; p < passes; ++p) {
    const int bits = (kbits - shift + passes - p - 1) / (passes - p);
    auto start = [&](int, uint32_t tot) {
      uint32_t all;
      return block_excl_scan<uint32_t>(tot, tmp, &all);
    };
    // the digits fit one round of threads (NT >= 256), so the scan spans them
    digit_places<NT, kSmallBits>(key, n, shift, bits, count, peers, start, place);
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (w * kWaveItems + i * kWave + l < n) {
        s_key[place[i]] = key[i];
        s_val[place[i]] = val[i];
      }
    __syncthreads();
    if (p + 1 < passes) {
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int x = w * kWaveItems + i * kWave + l;  // inside the stage; past n never used
        key[i] = s_key[x];
        val[i] = s_val[x];
      }
      __syncthreads();
    }
    shift += bits;
  }
  // thread t owns sorted places kRounds t ..: heads, their scan, the CSR
  const int p0 = threadIdx.x * kRounds;
  uint32_t heads = 0, live = 0;
  bool hd[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int p = p0 + k;
    const bool in = p < n && s_key[p] < (uint32_t)rows;
    hd[k] = in && (p == 0 || s_key[p - 1] != s_key[p]);
    heads += hd[k];
    live += in;
  }
  uint32_t U, valid;
  uint32_t u = block_excl_scan<uint32_t>(heads, tmp, &U);
  block_excl_scan<uint32_t>(live, tmp, &valid);
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int p = p0 + k;
    if (p >= (int)valid) break;
    u += hd[k];
    o.bm[p] = s_val[p];
    o.uid[p] = (int32_t)u - 1;
    if (hd[k]) {
      o.unique[u - 1] = s_key[p];
      o.seg[u - 1] = p;
    }
  }
  if (threadIdx.x == 0) write_totals(o, U, (int32_t)valid);
}

// ---------------------------------------------------------------- tiles
// Workgroups of 256 threads up to 64 tiles of 1024 tokens, of 1024 beyond:
// each sums the counts of the tiles before it, so tiles are few, but 16 of 4096
// leave the chip idle (16384 tokens: a scatter 9.0 us in tiles of 4096, 6.3 in
// tiles of 1024).
constexpr int kMidBits = 9;
constexpr int kMidBins = 1 << kMidBits;
constexpr int64_t kMidTiles = 64;
// Up to here the CSR counts the rows before a tile itself, beyond it a launch
// counts them first. Whole sorts with the recount / with the launch, of 32000
// rows: 8 tiles of 1024 22.7 / 23.2 us, 16 tiles 24.9 / 24.8, 24 tiles 26.4 /
// 25.9, 32 tiles 28.9 / 26.6, 64 tiles 38.3 / 31.4; 17 tiles of 4096 38.9 / 36.3,
// 64 tiles 59.5 / 41.0.
constexpr int64_t kRecountTiles = 16;
// Beyond this the dedup's passes sort. They take 58 to 62 us at 262144 tokens
// (32000 to 1000000 rows) where the tiles here take 41 to 58, and 80 to 85 at
// 1000000 tokens.
constexpr int64_t kMidMax = kMidTiles * 1024 * kRounds;  // 262144 tokens

template <bool kFirst>
__device__ __forceinline__ uint32_t load_key(const int64_t* ids, const uint32_t* keys, int32_t i,
                                             int64_t rows, int64_t padding, bool& bad) {
  if constexpr (kFirst) return token_key(ids[i], rows, padding, bad);
  return keys[i];
}

template <int NT, bool kFirst>
__global__ void __launch_bounds__(NT)
k_token_hist(const int64_t* __restrict__ ids, const uint32_t* __restrict__ keys, int32_t n,
             int64_t rows, int64_t padding, int shift, int bits, uint32_t* __restrict__ hist,
             int32_t* __restrict__ err) {
  __shared__ uint32_t h[kMidBins];
  for (int b = threadIdx.x; b < kMidBins; b += NT) h[b] = 0;
  __syncthreads();
  const uint32_t mask = (1u << bits) - 1;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int32_t x = (blockIdx.x * kRounds + i) * NT + threadIdx.x;
    if (x < n)
      atomicAdd(&h[(load_key<kFirst>(ids, keys, x, rows, padding, bad) >> shift) & mask], 1u);
  }
  if (kFirst) flag_err(err, bad, FS_EF_ID_RANGE);
  __syncthreads();
  for (uint32_t b = threadIdx.x; b <= mask; b += NT) hist[blockIdx.x * kMidBins + b] = h[b];
}

template <int NT, bool kFirst>
__global__ void __launch_bounds__(NT)
k_token_scatter(const int64_t* __restrict__ ids, const uint32_t* __restrict__ keys,
                const int32_t* __restrict__ vals, int32_t n, int64_t rows, int64_t padding,
                int shift, int bits, const uint32_t* __restrict__ hist, uint32_t* __restrict__ kout,
                int32_t* __restrict__ vout) {
  constexpr int kWaves = NT / kWave;
  constexpr int kParts = NT > kMidBins ? NT / kMidBins : 1;  // threads per digit
  __shared__ uint32_t count[kWaves][kMidBins];
  __shared__ uint64_t peers[kWaves][kMidBins];
  __shared__ uint32_t before[kParts][kMidBins], total[kParts][kMidBins];
  __shared__ uint32_t tmp[17];
  const int w = threadIdx.x / kWave, l = lane();
  const int32_t t0 = blockIdx.x * NT * kRounds, tiles = gridDim.x;
  uint32_t key[kRounds], place[kRounds];
  int32_t val[kRounds];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int32_t x = min(t0 + w * kWaveItems + i * kWave + l, n - 1);
    key[i] = load_key<kFirst>(ids, keys, x, rows, padding, bad);
    val[i] = kFirst ? x : vals[x];
  }
  for (int b = l; b < kMidBins; b += kWave) peers[w][b] = 0;
  // each digit's counts in the tiles before this one and in all of them
  for (int b = threadIdx.x % kMidBins; b < 1 << bits; b += NT) {
    const int part = threadIdx.x / kMidBins;
    uint32_t pre = 0, all = 0;
    for (int32_t t = part; t < tiles; t += 8 * kParts) {
      uint32_t v[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        v[y] = t + kParts * y < tiles ? hist[(t + kParts * y) * kMidBins + b] : 0u;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        all += v[y];
        if (t + kParts * y < (int32_t)blockIdx.x) pre += v[y];
      }
    }
    before[part][b] = pre;
    total[part][b] = all;
  }
  __syncthreads();
  uint32_t carry = 0;  // of the digits before this round's
  auto start = [&](int b, uint32_t) {
    uint32_t tot = 0, pre = 0, all;
    if (b < 1 << bits) {
#pragma unroll
      for (int y = 0; y < kParts; ++y) {
        tot += total[y][b];
        pre += before[y][b];
      }
    }
    const uint32_t ex = carry + block_excl_scan<uint32_t>(tot, tmp, &all);
    carry += all;
    return ex + pre;
  };
  digit_places<NT, kMidBits>(key, n - t0, shift, bits, count, peers, start, place);
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    if (t0 + w * kWaveItems + i * kWave + l < n) {
      kout[place[i]] = key[i];
      vout[place[i]] = val[i];
    }
}

// Heads of sorted places p0 .. p0 + 3 (bits), p0 a multiple of 4 that grows by
// 4 from lane to lane; *live: the places that hold a token that was not dropped
__device__ __forceinline__ uint32_t heads_of(const uint32_t* keys, int32_t p0, int32_t n,
                                             uint32_t rows, uint32_t* live) {
  uint32_t k[kRounds], bits = 0, in = 0;
  if (p0 + kRounds <= n) {
    const uint4 v = *(const uint4*)(keys + p0);
    k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
  } else {
#pragma unroll
    for (int y = 0; y < kRounds; ++y) k[y] = p0 + y < n ? keys[p0 + y] : rows;
  }
  uint32_t last = __shfl_up(k[kRounds - 1], 1, kWave);
  if (lane() == 0) last = p0 > 0 && p0 - 1 < n ? keys[p0 - 1] : rows;  // rows: no key of a row
#pragma unroll
  for (int y = 0; y < kRounds; ++y) {
    const bool ok = k[y] < rows;
    if (ok && last != k[y]) bits |= 1u << y;
    in += ok;
    last = k[y];
  }
  *live = in;
  return bits;
}

template <int NT>
__global__ void __launch_bounds__(NT)
k_token_heads(const uint32_t* __restrict__ keys, int32_t n, uint32_t rows,
              uint32_t* __restrict__ heads) {
  __shared__ uint32_t tmp[17];
  uint32_t live, tot;
  const uint32_t b = heads_of(keys, (blockIdx.x * NT + threadIdx.x) * kRounds, n, rows, &live);
  block_excl_scan<uint32_t>((uint32_t)popc(b), tmp, &tot);
  if (threadIdx.x == 0) heads[blockIdx.x] = tot;
}

// This thread's share of the heads in tiles 0 .. tiles - 1 (which are whole),
// eight tiles' keys in flight
template <int NT>
__device__ __forceinline__ uint32_t heads_before(const uint32_t* keys, uint32_t tiles,
                                                 uint32_t rows) {
  uint32_t sum = 0;
  for (uint32_t t = 0; t < tiles; t += 8) {
    uint4 v[8];
    uint32_t last[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const uint32_t p = ((t + y) * NT + threadIdx.x) * kRounds;
      v[y] = uint4{rows, rows, rows, rows};
      last[y] = rows;
      if (t + y < tiles) {
        v[y] = *(const uint4*)(keys + p);
        if (p > 0) last[y] = keys[p - 1];
      }
    }
#pragma unroll
    for (int y = 0; y < 8; ++y)
      sum += (uint32_t)(v[y].x < rows && v[y].x != last[y]) + (v[y].y < rows && v[y].y != v[y].x) +
             (v[y].z < rows && v[y].z != v[y].y) + (v[y].w < rows && v[y].w != v[y].z);
  }
  return sum;
}

// The CSR of one tile. `heads`: rows that begin in each tile; NULL: counted
// here over the tiles before this one.
template <int NT>
__global__ void __launch_bounds__(NT)
k_token_csr(const uint32_t* __restrict__ keys, int32_t n, uint32_t rows,
            const uint32_t* __restrict__ heads, SortOut o) {
  __shared__ uint64_t tmp64[17];
  uint32_t mine = 0, live;
  const int32_t p0 = (blockIdx.x * NT + threadIdx.x) * kRounds;
  const uint32_t b = heads_of(keys, p0, n, rows, &live);
  if (heads) {
    if (threadIdx.x < blockIdx.x) mine = heads[threadIdx.x];
  } else {
    mine = heads_before<NT>(keys, blockIdx.x, rows);
  }
  // three sums in one scan: heads before the tile (its total), heads and live
  // places before the thread (a tile has at most 4096 of each)
  uint64_t all;
  const uint64_t ex =
      block_excl_scan<uint64_t>((uint64_t)mine << 32 | (uint64_t)popc(b) << 16 | live, tmp64, &all);
  const uint32_t before = (uint32_t)(all >> 32), live_all = (uint32_t)all & 0xffffu;
  uint32_t u = before + ((uint32_t)(ex >> 16) & 0xffffu);
  const uint32_t tot = (uint32_t)(all >> 16) & 0xffffu;
#pragma unroll
  for (int y = 0; y < kRounds; ++y) {
    if (y >= (int)live) break;
    const int32_t p = p0 + y;
    if ((b >> y) & 1) {
      o.unique[u] = keys[p];
      o.seg[u] = p;
      ++u;
    }
    o.uid[p] = (int32_t)u - 1;
  }
  // the tile that holds the last token's place, or the first one if none is left
  const int32_t t0 = blockIdx.x * NT * kRounds, end = t0 + (int32_t)live_all;
  if (threadIdx.x == 0) {
    const bool last = live_all > 0 ? (end == n || keys[end] >= rows) : blockIdx.x == 0;
    if (last) write_totals(o, before + tot, end);
  }
}

// ---------------------------------------------------------------- large
// The tokens as the items of a one-shard batch with one more row.
__global__ void __launch_bounds__(kThreads)
k_token_items(const int64_t* __restrict__ ids, int64_t n, int64_t rows, int64_t padding,
              int64_t* __restrict__ keys, int32_t* __restrict__ bm, int64_t* __restrict__ bounds,
              int32_t* __restrict__ err) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  bool bad = false;
  if (i < n) {
    keys[i] = token_key(ids[i], rows, padding, bad);
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

// ---------------------------------------------------------------- host side
constexpr int64_t kSmall = 4096;  // tokens one workgroup sorts

int key_bits(uint64_t values) {  // of 0 .. values - 1
  int b = 1;
  while (b < 32 && (1ull << b) < values) ++b;
  return b;
}

size_t mid_bytes(int64_t n) {
  Carve c(nullptr);
  c.take<uint32_t>((size_t)n);
  c.take<uint32_t>((size_t)n);
  c.take<int32_t>((size_t)n);
  c.take<int32_t>((size_t)n);
  c.take<uint32_t>((size_t)(kMidTiles * kMidBins));
  c.take<uint32_t>((size_t)kMidTiles);
  return c.used + 256;
}

template <int NT>
int sort_mid(const int64_t* ids, int32_t n, int64_t rows, int64_t padding, int kbits,
             const SortOut& o, int32_t* err, void* ws, hipStream_t stream) {
  const int64_t tiles = cdiv(n, NT * kRounds);
  Carve c(ws);
  uint32_t* kbuf[2];
  int32_t* vbuf[2];
  for (auto& k : kbuf) k = c.take<uint32_t>((size_t)n);
  for (auto& v : vbuf) v = c.take<int32_t>((size_t)n);
  uint32_t* hist = c.take<uint32_t>((size_t)(kMidTiles * kMidBins));
  uint32_t* heads = c.take<uint32_t>((size_t)kMidTiles);
  const dim3 grid((unsigned)tiles), block(NT);
  const int passes = (kbits + kMidBits - 1) / kMidBits;
  for (int p = 0, shift = 0; p < passes; ++p) {
    const int bits = (kbits - shift + passes - p - 1) / (passes - p);
    const uint32_t* kin = kbuf[(p + 1) & 1];
    const int32_t* vin = vbuf[(p + 1) & 1];
    uint32_t* kout = kbuf[p & 1];
    int32_t* vout = p == passes - 1 ? o.bm : vbuf[p & 1];
    if (p == 0) {
      hipLaunchKernelGGL((k_token_hist<NT, true>), grid, block, 0, stream, ids, nullptr, n, rows,
                         padding, shift, bits, hist, err);
      FS_LAUNCH_CHECK();
      hipLaunchKernelGGL((k_token_scatter<NT, true>), grid, block, 0, stream, ids, nullptr, nullptr,
                         n, rows, padding, shift, bits, hist, kout, vout);
    } else {
      hipLaunchKernelGGL((k_token_hist<NT, false>), grid, block, 0, stream, nullptr, kin, n, rows,
                         padding, shift, bits, hist, nullptr);
      FS_LAUNCH_CHECK();
      hipLaunchKernelGGL((k_token_scatter<NT, false>), grid, block, 0, stream, nullptr, kin, vin, n,
                         rows, padding, shift, bits, hist, kout, vout);
    }
    FS_LAUNCH_CHECK();
    shift += bits;
  }
  const uint32_t* sorted = kbuf[(passes + 1) & 1];
  const bool recount = tiles <= kRecountTiles;
  if (!recount) {
    hipLaunchKernelGGL(k_token_heads<NT>, grid, block, 0, stream, sorted, n, (uint32_t)rows, heads);
    FS_LAUNCH_CHECK();
  }
  hipLaunchKernelGGL(k_token_csr<NT>, grid, block, 0, stream, sorted, n, (uint32_t)rows,
                     recount ? nullptr : heads, o);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_token_sort_workspace_size(int64_t n) {
  if (n <= kSmall) return 256;  // all in LDS
  const size_t mid = mid_bytes(std::min(n, kMidMax));
  if (n <= kMidMax) return mid;
  Carve c(nullptr);
  c.take<int64_t>((size_t)n);
  c.take<int32_t>((size_t)n);
  c.take<int64_t>(2);
  c.take<uint8_t>((size_t)n);
  return std::max(mid, c.used + 256 + fs_unique_workspace_size(n, 0, 1, 1));
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
  const SortOut o = {unique, unique_offsets, seg_offsets, occ_bm, occ_uid, counts};
  const int kbits = key_bits((uint64_t)rows + 1);

  if (n <= kSmall) {
    if (n <= 256 * kRounds)
      hipLaunchKernelGGL(k_token_sort_small<256>, dim3(1), dim3(256), 0, stream, ids, (int32_t)n,
                         rows, padding_id, kbits, o, err);
    else
      hipLaunchKernelGGL(k_token_sort_small<1024>, dim3(1), dim3(1024), 0, stream, ids, (int32_t)n,
                         rows, padding_id, kbits, o, err);
    FS_LAUNCH_CHECK();
    return FS_OK;
  }

  if (n <= kMidTiles * 256 * kRounds)
    return sort_mid<256>(ids, (int32_t)n, rows, padding_id, kbits, o, err, ws, stream);
  if (n <= kMidMax)
    return sort_mid<1024>(ids, (int32_t)n, rows, padding_id, kbits, o, err, ws, stream);

  Carve c(ws);
  int64_t* keys = c.take<int64_t>((size_t)n);
  int32_t* bm = c.take<int32_t>((size_t)n);
  int64_t* bounds = c.take<int64_t>(2);
  uint8_t* cls = c.take<uint8_t>((size_t)n);
  char* rest = (char*)ws + align_up(c.used, 256);
  hipLaunchKernelGGL(k_token_items, dim3((unsigned)cdiv(n, kThreads)), dim3(kThreads), 0, stream,
                     ids, n, rows, padding_id, keys, bm, bounds, err);
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
