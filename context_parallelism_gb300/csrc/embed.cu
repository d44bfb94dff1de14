// Token embedding with a factor, and its gradient.
//
//   h_i = scale w[t_i];   dw_v (+)= scale sum over {i : t_i = v} of dh_i, in order of i.
//
// Forward. Bound: HBM (the rows that occur are read, h is written): 131072 tokens of 4096 features in
// 225 us, 90 % of a copy's rate. A warp moves 1024 features of one token, four 16-byte vectors a lane,
// and streams them out past the rows that L2 keeps (2 % faster than plain stores; two vectors a lane
// 232 us, eight 225).
//
// Backward. The places are sorted by token, stably, so that each row of dw is one sum of rows of dh in
// the order of the sequence: no atomic float additions, the same bits every time. The sorted places
// are cut into chunks of equal length whatever the tokens' counts (the commonest token of a text may
// have thousands of places, most have one or none): a chunk adds up its rows run by run. A run that
// lies inside the chunk goes straight to dw; what belongs to a run that goes on beside the chunk is
// left as a partial sum, at most two a chunk, and a last kernel joins them in order. Rows of tokens
// that do not occur are zeroed by blocks of the same launch, from a bitmap that the sort leaves. (Some
// of them zeroed beside the sort instead: no gain at 4097 places, 10 us lost at 8192, whose tokens then
// wait behind the stores.)
//
// Sort, up to kSmall places: one launch that counts, for each place, the keys before it. That is S^2
// comparisons, yet 6 us for 4097 places and 13 for 8192 over all SMs, where a radix sort in the shared
// memory of one block took 18 and 22, and its launches on all SMs 22 (at 10240 places: 16, against 20).
// More: a stable radix sort of 32-bit tokens with their places, in passes of up to 9 bits (17 bits of
// vocabulary: 2 passes), two launches a pass, histograms of 2048 places and scatter, each scatter block
// adding up the histograms before it (with more than kFewTiles blocks a launch between does that). A
// place's rank in its block: warps count 32 places at a time, matching equal digits by ballots.
#include "internal.h"
#include "rope.cuh"

namespace upipe {
namespace {

constexpr int kEmbedClass = 17;
constexpr int kTile = 2048;  // places of a sort block
constexpr int kFewTiles = 96;  // (512 tiles, 2^20 places: 352 us, 400 where each block adds them up)
constexpr int kSortThreads = 256;
constexpr int kRounds = kTile / kSortThreads;
constexpr int kWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;

// ---- forward ----------------------------------------------------------------------------------

constexpr int kVecs = 4;  // vectors a lane
constexpr int kFwdThreads = 256;

__global__ void __launch_bounds__(kFwdThreads)
    embed_kernel(const int64_t* __restrict__ tokens, const uint4* __restrict__ w,
                 uint4* __restrict__ h, int64_t S, int vecs, int64_t V, float scale, int parts) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
  const int64_t i = div_fl(unit, parts);
  if (i >= S) return;
  const int v0 = static_cast<int>(unit - i * parts) * (32 * kVecs) + (threadIdx.x & 31);
  const int64_t t = tokens[i];
  uint4 x[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int v = v0 + 32 * j;
    x[j] = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < V && v < vecs) x[j] = __ldg(w + t * vecs + v);
  }
  const uint32_t nan2 = 0x7fc07fc0u;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int v = v0 + 32 * j;
    if (v >= vecs) break;
    if (t >= V) {
      x[j] = make_uint4(nan2, nan2, nan2, nan2);
    } else if (scale != 1.f) {
      float f[8];
      unpack_bf16x8(x[j], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= scale;
      x[j] = pack_bf16x8(f);
    }
    __stcs(h + i * vecs + v, x[j]);
  }
}

// ---- sort -------------------------------------------------------------------------------------

// Key of place i in the first pass: its token, or V (sorted behind all) where that names no row.
__device__ __forceinline__ uint32_t first_key(const EmbedArgs& a, int64_t i) {
  const int64_t t = a.tokens[i];
  return static_cast<uint32_t>(t >= 0 && t < a.V ? t : a.V);
}

// The bitmap's bit of a key that is a token (the commonest ones are set already).
__device__ __forceinline__ void mark_present(const EmbedArgs& a, uint32_t key) {
  if (!a.present || key >= static_cast<uint32_t>(a.V)) return;
  uint32_t* word = a.present + (key >> 5);
  const uint32_t bit = 1u << (key & 31);
  if (!(*reinterpret_cast<volatile uint32_t*>(word) & bit)) atomicOr(word, bit);
}

// Lanes with this lane's digit (bits wide), among `active`.
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, int bits, uint32_t active) {
  uint32_t same = active;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xffffffffu, (digit >> b) & 1);
    same &= (digit >> b) & 1 ? set : ~set;
  }
  return same;
}

// Rank of each of a warp's places among those before it with its digit: place r of lane l comes after
// all places of smaller r, and of smaller l in its own. count (one per digit, zeros before) ends as the
// warp's histogram.
template <int rounds>
__device__ __forceinline__ void warp_ranks(const uint32_t (&digit)[rounds], uint32_t n, int bits,
                                           uint32_t* count, uint32_t (&rank)[rounds]) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < rounds; ++r) {
    if (r * 32 >= n) break;
    const bool in = r * 32 + lane < n;
    const uint32_t same = same_digit(digit[r], bits, __ballot_sync(0xffffffffu, in));
    uint32_t before = 0;
    if (in) before = count[digit[r]];
    __syncwarp();
    rank[r] = before + __popc(same & ((1u << lane) - 1));
    if (in && (same >> lane) == 1) count[digit[r]] = before + __popc(same);
    __syncwarp();
  }
}

// Exclusive sums of x over the block's threads (a multiple of 32, at most 1024).
__device__ __forceinline__ uint32_t block_before(uint32_t x, uint32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t up = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, up, m);
    if (lane >= m) up += o;
  }
  if (lane == 31) warp_sum[warp] = up;
  __syncthreads();
  uint32_t before = up - x;
  for (int k = 0; k < warp; ++k) before += warp_sum[k];
  __syncthreads();
  return before;
}

// Up to kSmall places are sorted by counting, for each, the keys before it: a warp takes two places, and
// every block has all keys in shared memory. With them it also makes its part of the bitmap.
constexpr int kSmall = 8192;
constexpr int kRankThreads = 512;
constexpr int kRankBlocks = 152;
constexpr int kRankWords = 2048;  // of the bitmap at a time

__global__ void __launch_bounds__(kRankThreads) rank_kernel(const EmbedArgs a, uint32_t* keys_out,
                                                            uint32_t* places_out) {
  extern __shared__ uint4 quad[];
  __shared__ uint32_t word[kRankWords];
  uint32_t* key = reinterpret_cast<uint32_t*>(quad);
  launch_dependents();
  const int n = static_cast<int>(a.S), quads = (n + 3) / 4;
#pragma unroll 8
  for (int i = threadIdx.x; i < 4 * quads; i += kRankThreads)
    key[i] = i < n ? first_key(a, i) : 0xffffffffu;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (n + kRankBlocks - 1) / kRankBlocks;
  const int lo = blockIdx.x * per, hi = min(lo + per, n);
  for (int i = lo + 2 * warp; i < hi; i += kRankThreads / 16) {
    const int j = min(i + 1, hi - 1);
    const uint32_t ki = key[i], kj = key[j];
    const int qi = i >> 2, qj = j >> 2;
    uint32_t ci = 0, cj = 0;
#pragma unroll 4
    for (int q = lane; q < quads; q += 32) {
      const uint4 x = quad[q];
      const uint32_t ti = ki + (q < qi), tj = kj + (q < qj);  // equal keys count where they come before
      ci += (x.x < ti) + (x.y < ti) + (x.z < ti) + (x.w < ti);
      cj += (x.x < tj) + (x.y < tj) + (x.z < tj) + (x.w < tj);
    }
    if (lane < (i & 3)) ci += key[4 * qi + lane] == ki;
    if (lane < (j & 3)) cj += key[4 * qj + lane] == kj;
    ci = __reduce_add_sync(0xffffffffu, ci);
    cj = __reduce_add_sync(0xffffffffu, cj);
    if (lane < 2) {  // (the same place twice at the end)
      const uint32_t to = lane ? cj : ci;
      keys_out[to] = lane ? kj : ki;
      places_out[to] = lane ? j : i;
    }
  }
  if (!a.present) return;
  const int64_t words = (a.V + 31) / 32, some = (words + kRankBlocks - 1) / kRankBlocks;
  const int64_t first = blockIdx.x * some, end = first + some < words ? first + some : words;
  for (int64_t w0 = first; w0 < end; w0 += kRankWords) {
    const uint32_t len = static_cast<uint32_t>(end - w0 < kRankWords ? end - w0 : kRankWords);
    for (uint32_t k = threadIdx.x; k < len; k += kRankThreads) word[k] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRankThreads) {
      const uint32_t at = (key[i] >> 5) - static_cast<uint32_t>(w0);  // (those before: large)
      if (at < len) atomicOr(&word[at], 1u << (key[i] & 31));
    }
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < len; k += kRankThreads) a.present[w0 + k] = word[k];
    __syncthreads();
  }
}

// hist[tile][digit]; the first pass marks the tokens that occur (present: zeros before).
template <bool kFirst>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const EmbedArgs a,
                                                                  const uint32_t* keys, int shift,
                                                                  int bins) {
  __shared__ uint32_t count[kMaxBins];
  launch_dependents();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) count[d] = 0;
  if (!kFirst) grid_dependency_wait();
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
  uint32_t key[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kSortThreads + threadIdx.x;
    key[r] = i >= a.S ? 0 : kFirst ? first_key(a, i) : keys[i];
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (base + r * kSortThreads + threadIdx.x >= a.S) break;
    atomicAdd(&count[(key[r] >> shift) & (bins - 1)], 1u);
    if (kFirst) mark_present(a, key[r]);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads)
    a.hist[static_cast<int64_t>(blockIdx.x) * bins + d] = count[d];
}

// With many tiles: hist[tile][digit] becomes the places before the tile of that digit, and hist[tiles] the
// digits' totals. A block takes 16 digits, 16 threads each with a run of the tiles.
__global__ void __launch_bounds__(256) sort_scan_kernel(uint32_t* hist, int64_t tiles, int bins) {
  __shared__ uint32_t sum[16][16];
  launch_dependents();
  grid_dependency_wait();
  const int d = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
  const int64_t per = (tiles + 15) / 16, lo = part * per, hi = lo + per < tiles ? lo + per : tiles;
  uint32_t total = 0;
  if (d < bins) {
#pragma unroll 8
    for (int64_t t = lo; t < hi; ++t) total += hist[t * bins + d];
  }
  sum[part][threadIdx.x & 15] = total;
  __syncthreads();
  if (d >= bins) return;
  uint32_t at = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t c = sum[k][threadIdx.x & 15];
    if (k < part) at += c;
    all += c;
  }
#pragma unroll 8
  for (int64_t t = lo; t < hi; ++t) {
    const uint32_t c = hist[t * bins + d];
    hist[t * bins + d] = at;
    at += c;
  }
  if (part == 0) hist[tiles * bins + d] = all;
}

template <bool kFirst>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const EmbedArgs a,
                                                                    const uint32_t* keys,
                                                                    const uint32_t* places,
                                                                    uint32_t* keys_out,
                                                                    uint32_t* places_out, int shift,
                                                                    int bits, int scanned) {
  __shared__ uint32_t count[kWarps][kMaxBins];
  __shared__ uint32_t warp_sum[32];
  launch_dependents();
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = threadIdx.x; d < kWarps * bins; d += kSortThreads) count[d >> bits][d & (bins - 1)] = 0;
  grid_dependency_wait();
  __syncthreads();
  // a warp owns kTile / kWarps places in a row
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile + warp * (kTile / kWarps);
  uint32_t key[kRounds], place[kRounds], digit[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 32 + lane;
    const bool in = i < a.S;
    key[r] = !in ? 0u : kFirst ? first_key(a, i) : keys[i];
    place[r] = !in ? 0u : kFirst ? static_cast<uint32_t>(i) : places[i];
  }
  // places before this tile's of each digit: two digits a thread (bins: at most 2 kSortThreads)
  uint32_t at[2] = {0, 0}, total[2] = {0, 0};
  if (2 * static_cast<int>(threadIdx.x) < bins) {  // (bins is even)
    const uint2* hist = reinterpret_cast<const uint2*>(a.hist) + threadIdx.x;
    const int row = bins / 2, self = blockIdx.x;
    if (scanned) {
      const uint2 c = hist[static_cast<int64_t>(self) * row], all = hist[static_cast<int64_t>(gridDim.x) * row];
      at[0] = c.x;
      at[1] = c.y;
      total[0] = all.x;
      total[1] = all.y;
    } else {
#pragma unroll 16
      for (int t = 0; t < static_cast<int>(gridDim.x); ++t) {
        const uint2 c = hist[t * row];
        if (t < self) {
          at[0] += c.x;
          at[1] += c.y;
        }
        total[0] += c.x;
        total[1] += c.y;
      }
    }
  }
  const uint32_t start = block_before(total[0] + total[1], warp_sum);
  at[0] += start;
  at[1] += start + total[0];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) digit[r] = (key[r] >> shift) & (bins - 1);
  const int64_t left = a.S - base;
  const uint32_t mine = left < 0 ? 0 : left < kTile / kWarps ? left : kTile / kWarps;
  warp_ranks<kRounds>(digit, mine, bits, count[warp], rank);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = 2 * threadIdx.x + k;
    if (d >= bins) continue;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t n = count[w][d];
      count[w][d] = at[k];
      at[k] += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (r * 32 + lane >= mine) break;
    const uint32_t to = count[warp][digit[r]] + rank[r];
    keys_out[to] = key[r];
    places_out[to] = place[r];
  }
}

// ---- sums -------------------------------------------------------------------------------------

// Eight elements of a row of dw, from a sum over its places.
__device__ __forceinline__ void put_row(const EmbedArgs& a, uint32_t key, int f, const float (&s)[8]) {
  float4* dst = reinterpret_cast<float4*>(a.dw + static_cast<int64_t>(key) * a.Dm + f);
  float4 u = make_float4(s[0] * a.scale, s[1] * a.scale, s[2] * a.scale, s[3] * a.scale);
  float4 v = make_float4(s[4] * a.scale, s[5] * a.scale, s[6] * a.scale, s[7] * a.scale);
  if (a.add) {
    const float4 x = dst[0], y = dst[1];
    u = make_float4(u.x + x.x, u.y + x.y, u.z + x.z, u.w + x.w);
    v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
  }
  __stcs(dst, u);
  __stcs(dst + 1, v);
}

__device__ __forceinline__ float* part_at(const EmbedArgs& a, int64_t chunk, int which, int f) {
  return a.part + (chunk * 2 + which) * a.Dm + f;
}

// Blocks [0, chunks * slices): one slice of features of one chunk of the sorted places. The others:
// rows of dw whose token does not occur, zero_rows each.
// (131072 places of 4096 features: 499 to 506 us with a row a block, 517 with 16; 16384 of 256: 52, 65 with
// 4 rows)
constexpr int kZeroBytes = 16384;
constexpr int kMaxChunk = 128;
constexpr int kAhead = 8;  // rows of dh in flight a thread

__global__ void __launch_bounds__(128) embed_sum_kernel(const EmbedArgs a, const uint32_t* keys,
                                                        const uint32_t* places) {
  __shared__ uint32_t key[kMaxChunk + 2], place[kMaxChunk];
  grid_dependency_wait();
  launch_dependents();  // here, so that the next kernel has the sorted keys from its start
  const int64_t units = a.chunks * a.slices;
  if (static_cast<int64_t>(blockIdx.x) >= units) {
    const int64_t v0 = (static_cast<int64_t>(blockIdx.x) - units) * a.zero_rows;
    const uint32_t present = a.present[v0 >> 5] >> (v0 & 31);  // (they share a word)
    for (int r = 0; r < a.zero_rows && v0 + r < a.V; ++r) {
      if (present >> r & 1) continue;
      float4* dst = reinterpret_cast<float4*>(a.dw + (v0 + r) * a.Dm);
      for (int k = threadIdx.x; k < a.Dm / 4; k += blockDim.x)
        __stcs(dst + k, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    return;
  }
  const int64_t chunk = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - chunk * a.slices);
  const int64_t lo = chunk * a.chunk;
  const int n = static_cast<int>(a.S - lo < a.chunk ? a.S - lo : a.chunk);
  // key[0] and key[n + 1]: the neighbours beside the chunk (none: a key that no row has)
  for (int k = threadIdx.x; k < n + 2; k += blockDim.x) {
    const int64_t i = lo + k - 1;
    key[k] = i >= 0 && i < a.S ? keys[i] : 0xffffffffu;
    if (k >= 1 && k <= n) place[k - 1] = places[i];
  }
  __syncthreads();
  const int f = (slice * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
  if (f >= a.Dm) return;
  const uint32_t none = static_cast<uint32_t>(a.V);
  const __nv_bfloat16* dh = a.dh + f;
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f;
  bool open = key[0] == key[1];  // the run goes on from the chunk before
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j < n && key[i0 + j + 1] < none)
        x[j] = __ldcs(reinterpret_cast<const uint4*>(dh + static_cast<int64_t>(place[i0 + j]) * a.Dm));
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j;
      if (i >= n) break;
      const uint32_t k = key[i + 1];
      if (k >= none) return;  // sorted last: places without a row
      float y[8];
      unpack_bf16x8(x[j], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += y[e];
      if (i + 1 < n && key[i + 2] == k) continue;
      // the run ends here, or goes on in the next chunk
      const bool goes_on = key[i + 2] == k;
      if (open || goes_on) {
        float4* dst = reinterpret_cast<float4*>(part_at(a, chunk, open ? 0 : 1, f));
        dst[0] = make_float4(s[0], s[1], s[2], s[3]);
        dst[1] = make_float4(s[4], s[5], s[6], s[7]);
      } else {
        put_row(a, k, f, s);
      }
      open = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = 0.f;
    }
  }
}

// One block for each chunk in which a run begins that goes on: its partial sums, kJoin runs of chunks one
// beside the other (a token that fills a tenth of a long sequence has hundreds), then these in order.
// Which runs these are it finds while the last sums are made (1 us less).
constexpr int kJoin = 4;
__global__ void __launch_bounds__(128 * kJoin) embed_join_kernel(const EmbedArgs a,
                                                                 const uint32_t* keys) {
  __shared__ float4 sums[kJoin - 1][2][128];
  const int64_t chunk = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - chunk * a.slices);
  const int64_t lo = chunk * a.chunk, hi = lo + a.chunk;
  uint32_t k = 0xffffffffu, next = 0, before = k;
  if (hi < a.S) {  // not the last chunk
    k = __ldcg(keys + hi - 1);
    next = __ldcg(keys + hi);
    if (lo > 0) before = __ldcg(keys + lo - 1);
  }
  if (k >= static_cast<uint32_t>(a.V) || next != k || before == k) {  // (before: it began there)
    // What comes behind this launch in a stream or a graph waits for it alone, so it must not end before
    // the sums do, also where no block has anything to join: the first block always waits for them, and
    // with it the launch. (All blocks: 8192 places of 4096 features added to dw 51.7 us, so 50.3.)
    if (blockIdx.x == 0) grid_dependency_wait();
    return;
  }
  // the last chunk that it reaches: the keys are sorted, so those that begin with it come first
  int64_t last = chunk;
  for (int more = blockDim.x; more == static_cast<int>(blockDim.x); last += more) {
    const int64_t i = (last + 1 + threadIdx.x) * a.chunk;
    more = __syncthreads_count(i < a.S && __ldcg(keys + i) == k);
  }
  grid_dependency_wait();
  const int threads = blockDim.x / kJoin, part = threadIdx.x / threads,
            col = threadIdx.x - part * threads;
  const int f = (slice * threads + col) * 8;
  const bool in = f < a.Dm;
  const int64_t per = (last - chunk + kJoin) / kJoin;  // partial sums of a part, the chunk's own first
  const int64_t from = chunk + part * per, to = from + per - 1 < last ? from + per - 1 : last;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  if (in) {
#pragma unroll 8
    for (int64_t c = from; c <= to; ++c) {
      const float4* p = reinterpret_cast<const float4*>(part_at(a, c, c == chunk ? 1 : 0, f));
      const float4 x = p[0], y = p[1];
      s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
      s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
    }
    if (part > 0) {
      sums[part - 1][0][col] = make_float4(s[0], s[1], s[2], s[3]);
      sums[part - 1][1][col] = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
  __syncthreads();
  if (part > 0 || !in) return;
#pragma unroll
  for (int p = 0; p < kJoin - 1; ++p) {
    const float4 x = sums[p][0][col], y = sums[p][1][col];
    s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
    s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
  }
  put_row(a, k, f, s);
}

}  // namespace

EmbedPlan plan_embed(int64_t S, int Dm, int64_t V) {
  EmbedPlan p{};
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // keys 0 .. V
  p.passes = (bits + 8) / 9;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = S <= kSmall ? 0 : (S + kTile - 1) / kTile;
  const int vecs = Dm / 8;
  p.threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  p.slices = (vecs + p.threads - 1) / p.threads;
  // chunks: as long as an equal share of whole rounds of 1216 blocks, those of 128 threads that are resident
  // (8 on each of 152 SMs), so that the last round is full and partial sums (two a chunk) stay few: 32768
  // places of 4096 features 208 us, 218 with powers of two and at least twice as many chunks. More of the
  // narrower blocks of fewer features are resident, yet rounds of as many, with shorter chunks, are worse
  // for most sizes (256 features, 32 threads a block, rounds of 1216 and of 4864: 32768 places 46.6 and
  // 65.2 us, 16384 45.7 and 50.5, 131072 88.5 and 84.4).
  const int64_t all = S * p.slices, round = 1216, rounds = (all + round * kMaxChunk - 1) / (round * kMaxChunk);
  p.chunk = static_cast<int>((all + round * rounds - 1) / (round * rounds));
  if (p.chunk < 8) p.chunk = 8;
  p.chunks = (S + p.chunk - 1) / p.chunk;
  p.zero_rows = 32;
  while (p.zero_rows > 1 && int64_t(p.zero_rows) * Dm * 4 > kZeroBytes) p.zero_rows /= 2;
  p.blocks = p.chunks * p.slices + (V + p.zero_rows - 1) / p.zero_rows;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = take(static_cast<size_t>(S) * 4);
    p.places[i] = take(static_cast<size_t>(S) * 4);
  }
  p.hist = take(static_cast<size_t>(p.tiles + 1) * (size_t(1) << p.bits) * 4);
  p.present = take(static_cast<size_t>((V + 31) / 32) * 4);
  p.part = take(static_cast<size_t>(p.chunks) * 2 * Dm * 4);
  p.total = off;
  return p;
}

cudaError_t launch_embed(const int64_t* tokens, const void* w, void* h, int64_t S, int Dm,
                         int64_t V, float scale, cudaStream_t stream) {
  const int vecs = Dm / 8, parts = (vecs + 32 * kVecs - 1) / (32 * kVecs);
  const int64_t units = S * parts;
  launch_begin(kEmbedClass, stream);
  constexpr int kUnits = kFwdThreads / 32;
  embed_kernel<<<static_cast<unsigned>((units + kUnits - 1) / kUnits), kFwdThreads, 0, stream>>>(
      tokens, static_cast<const uint4*>(w), static_cast<uint4*>(h), S, vecs, V, scale, parts);
  const cudaError_t e = cudaGetLastError();
  launch_end(kEmbedClass, stream);
  return e;
}

cudaError_t launch_embed_bwd(EmbedArgs a, const EmbedPlan& p, uint8_t* ws, cudaStream_t stream) {
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + p.keys[0]),
                       reinterpret_cast<uint32_t*>(ws + p.keys[1])};
  uint32_t* places[2] = {reinterpret_cast<uint32_t*>(ws + p.places[0]),
                         reinterpret_cast<uint32_t*>(ws + p.places[1])};
  a.hist = reinterpret_cast<uint32_t*>(ws + p.hist);
  a.present = a.add ? nullptr : reinterpret_cast<uint32_t*>(ws + p.present);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.slices = p.slices;
  const int bins = 1 << p.bits;
  cudaError_t e = cudaSuccess;
  auto launch = [&](auto kernel, int64_t grid, int block, size_t smem, bool early, auto... args) {
    if (e != cudaSuccess) return;
    launch_begin(kEmbedClass, stream);
    e = launch_after(kernel, dim3(static_cast<unsigned>(grid)), dim3(block), smem, stream, early,
                     args...);
    launch_end(kEmbedClass, stream);
  };
  int in = 0;
  if (p.tiles == 0) {
    launch(rank_kernel, kRankBlocks, kRankThreads, static_cast<size_t>(a.S + 3) / 4 * 16, false, a,
           keys[0], places[0]);
  } else {
    if (a.present) e = cudaMemsetAsync(a.present, 0, static_cast<size_t>((a.V + 31) / 32) * 4, stream);
    const int scanned = p.tiles > kFewTiles;
    for (int pass = 0; pass < p.passes; ++pass, in ^= 1) {
      const int shift = pass * p.bits;
      const uint32_t *k = keys[in], *pl = places[in];
      if (pass == 0)
        launch(sort_count_kernel<true>, p.tiles, kSortThreads, 0, false, a, k, shift, bins);
      else
        launch(sort_count_kernel<false>, p.tiles, kSortThreads, 0, true, a, k, shift, bins);
      if (scanned) launch(sort_scan_kernel, (bins + 15) / 16, 256, 0, true, a.hist, p.tiles, bins);
      if (pass == 0)
        launch(sort_scatter_kernel<true>, p.tiles, kSortThreads, 0, true, a, k, pl, keys[in ^ 1],
               places[in ^ 1], shift, p.bits, scanned);
      else
        launch(sort_scatter_kernel<false>, p.tiles, kSortThreads, 0, true, a, k, pl, keys[in ^ 1],
               places[in ^ 1], shift, p.bits, scanned);
    }
  }
  a.zero_rows = p.zero_rows;
  const uint32_t *k = keys[in], *pl = places[in];
  launch(embed_sum_kernel, a.present ? p.blocks : p.chunks * p.slices, p.threads, 0, true, a, k, pl);
  if (p.chunks > 1) launch(embed_join_kernel, p.chunks * p.slices, p.threads * kJoin, 0, true, a, k);
  return e;
}

}  // namespace upipe
