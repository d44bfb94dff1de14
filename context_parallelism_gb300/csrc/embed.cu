// Token embedding with a factor, and its gradient.
//
//   h_i = scale w[t_i];   dw_v (+)= scale sum over {i : t_i = v} of dh_i, in order of i.
//
// Forward. Bound: HBM (the rows that occur are read, h is written). A warp moves 1024 features of one
// token, four 16-byte vectors a lane, and streams them out past the rows that L2 keeps.
//
// Backward. The places are sorted by token, stably, so that each row of dw is one sum of rows of dh in
// the order of the sequence: no atomic float additions, the same bits every time. The sorted places
// are cut into chunks of equal length whatever the tokens' counts (the commonest token of a text may
// have thousands of places, most have one or none): a chunk adds up its rows run by run. A run that
// lies inside the chunk goes straight to dw; what belongs to a run that goes on beside the chunk is
// left as a partial sum, at most two a chunk, and a last kernel joins them in order. Rows of tokens
// that do not occur are zeroed by blocks of the same launch, from a bitmap that the sort leaves.
//
// Sort: a stable radix sort of 32-bit tokens with their places, in passes of up to 9 bits (17 bits of
// vocabulary: 2 passes), three small launches a pass: histograms of 4096 places, one scan, scatter.
// A place's rank in its block: warps count 32 places at a time, matching equal digits by ballots.
#include "internal.h"
#include "rope.cuh"

namespace upipe {
namespace {

constexpr int kEmbedClass = 17;
constexpr int kTile = 4096;  // places of a sort block
constexpr int kSortThreads = 256;
constexpr int kRounds = kTile / kSortThreads;
constexpr int kWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;

// ---- forward ----------------------------------------------------------------------------------

__global__ void __launch_bounds__(256) embed_kernel(const int64_t* __restrict__ tokens,
                                                    const uint4* __restrict__ w,
                                                    uint4* __restrict__ h, int64_t S, int vecs,
                                                    int64_t V, float scale, int parts) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t i = div_fl(unit, parts);
  if (i >= S) return;
  const int v0 = static_cast<int>(unit - i * parts) * 128 + (threadIdx.x & 31);
  const int64_t t = tokens[i];
  uint4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int v = v0 + 32 * j;
    x[j] = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < V && v < vecs) x[j] = __ldg(w + t * vecs + v);
  }
  const uint32_t nan2 = 0x7fc07fc0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
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

template <bool kFirst>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const EmbedArgs a,
                                                                  const uint32_t* keys, int shift,
                                                                  int bins) {
  __shared__ uint32_t count[kMaxBins];
  launch_dependents();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) count[d] = 0;
  if (!kFirst) grid_dependency_wait();
  if (kFirst && a.present) {
    const int64_t words = (a.V + 31) / 32;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; k < words;
         k += static_cast<int64_t>(gridDim.x) * kSortThreads)
      a.present[k] = 0;
  }
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
#pragma unroll 4
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kSortThreads + threadIdx.x;
    if (i >= a.S) break;
    const uint32_t key = kFirst ? first_key(a, i) : keys[i];
    atomicAdd(&count[(key >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads)
    a.hist[static_cast<int64_t>(d) * gridDim.x + blockIdx.x] = count[d];
}

// Exclusive sums of hist[n] in place, one block.
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* hist, int64_t n) {
  __shared__ uint32_t warp_sum[32];
  __shared__ uint32_t carry;
  launch_dependents();
  if (threadIdx.x == 0) carry = 0;
  grid_dependency_wait();
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t base = 0; base < n; base += 4096) {
    const int64_t i = base + 4 * threadIdx.x;
    uint32_t x[4], s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = i + j < n ? hist[i + j] : 0;
      s += x[j];
    }
    uint32_t up = s;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, up, m);
      if (lane >= m) up += o;
    }
    if (lane == 31) warp_sum[warp] = up;
    __syncthreads();
    uint32_t before = carry;
    for (int k = 0; k < warp; ++k) before += warp_sum[k];
    uint32_t at = before + up - s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j < n) hist[i + j] = at;
      at += x[j];
    }
    __syncthreads();
    if (threadIdx.x == 1023) carry = at;
    __syncthreads();
  }
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

template <bool kFirst>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const EmbedArgs a,
                                                                    const uint32_t* keys,
                                                                    const uint32_t* places,
                                                                    uint32_t* keys_out,
                                                                    uint32_t* places_out, int shift,
                                                                    int bits) {
  __shared__ uint32_t count[kWarps][kMaxBins];
  launch_dependents();
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = threadIdx.x; d < kWarps * bins; d += kSortThreads) count[d / bins][d % bins] = 0;
  grid_dependency_wait();
  __syncthreads();
  // a warp owns 512 places in a row
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile + warp * (kTile / kWarps);
  uint32_t key[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 32 + lane;
    const bool in = i < a.S;
    key[r] = !in ? 0u : kFirst ? first_key(a, i) : keys[i];
    const uint32_t digit = (key[r] >> shift) & (bins - 1);
    const uint32_t active = __ballot_sync(0xffffffffu, in);
    const uint32_t same = same_digit(digit, bits, active);
    uint32_t before = 0;
    if (in) before = count[warp][digit];
    __syncwarp();
    rank[r] = before + __popc(same & ((1u << lane) - 1));
    if (in && (same >> lane) == 1) count[warp][digit] = before + __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) {
    uint32_t at = a.hist[static_cast<int64_t>(d) * gridDim.x + blockIdx.x];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const uint32_t n = count[k][d];
      count[k][d] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 32 + lane;
    if (i >= a.S) break;
    const uint32_t at = count[warp][(key[r] >> shift) & (bins - 1)] + rank[r];
    keys_out[at] = key[r];
    places_out[at] = kFirst ? static_cast<uint32_t>(i) : places[i];
    if (kFirst && a.present && key[r] < static_cast<uint32_t>(a.V)) {
      uint32_t* word = a.present + (key[r] >> 5);
      const uint32_t bit = 1u << (key[r] & 31);
      if (!(*reinterpret_cast<volatile uint32_t*>(word) & bit)) atomicOr(word, bit);
    }
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
// rows of dw whose token does not occur, kZeroRows each.
constexpr int kZeroRows = 16;
constexpr int kMaxChunk = 128;
constexpr int kAhead = 8;  // rows of dh in flight a thread

__global__ void __launch_bounds__(128) embed_sum_kernel(const EmbedArgs a, const uint32_t* keys,
                                                        const uint32_t* places) {
  __shared__ uint32_t key[kMaxChunk + 2], place[kMaxChunk];
  launch_dependents();
  grid_dependency_wait();
  const int64_t units = a.chunks * a.slices;
  if (static_cast<int64_t>(blockIdx.x) >= units) {
    const int64_t v0 = (static_cast<int64_t>(blockIdx.x) - units) * kZeroRows;
    for (int r = 0; r < kZeroRows && v0 + r < a.V; ++r) {
      const int64_t v = v0 + r;
      if (a.present[v >> 5] >> (v & 31) & 1) continue;
      float4* dst = reinterpret_cast<float4*>(a.dw + v * a.Dm);
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

// One block for each chunk in which a run begins that goes on: its partial sums in order.
__global__ void __launch_bounds__(128) embed_join_kernel(const EmbedArgs a, const uint32_t* keys) {
  launch_dependents();
  grid_dependency_wait();
  const int64_t chunk = blockIdx.x / a.slices;
  const int slice = static_cast<int>(blockIdx.x - chunk * a.slices);
  const int64_t lo = chunk * a.chunk, hi = lo + a.chunk;
  if (hi >= a.S) return;  // the last chunk
  const uint32_t k = keys[hi - 1];
  if (k >= static_cast<uint32_t>(a.V) || keys[hi] != k) return;
  if (lo > 0 && keys[lo - 1] == k) return;  // it began before
  const int f = (slice * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
  if (f >= a.Dm) return;
  float s[8];
  const float4* first = reinterpret_cast<const float4*>(part_at(a, chunk, 1, f));
  const float4 u = first[0], v = first[1];
  s[0] = u.x; s[1] = u.y; s[2] = u.z; s[3] = u.w;
  s[4] = v.x; s[5] = v.y; s[6] = v.z; s[7] = v.w;
  for (int64_t c = chunk + 1; c * a.chunk < a.S && keys[c * a.chunk] == k; ++c) {
    const float4* p = reinterpret_cast<const float4*>(part_at(a, c, 0, f));
    const float4 x = p[0], y = p[1];
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
  p.tiles = (S + kTile - 1) / kTile;
  const int vecs = Dm / 8;
  p.threads = vecs >= 128 ? 128 : (vecs + 31) / 32 * 32;
  p.slices = (vecs + p.threads - 1) / p.threads;
  // chunks: long enough that their partial sums (two a chunk) cost little, short enough for some
  // 16 blocks on each of 152 SMs
  p.chunk = kMaxChunk;
  while (p.chunk > 8 && S * p.slices < static_cast<int64_t>(p.chunk) * 2432) p.chunk /= 2;
  p.chunks = (S + p.chunk - 1) / p.chunk;
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
  p.hist = take(static_cast<size_t>(p.tiles) * (size_t(1) << p.bits) * 4);
  p.present = take(static_cast<size_t>((V + 31) / 32) * 4);
  p.part = take(static_cast<size_t>(p.chunks) * 2 * Dm * 4);
  p.total = off;
  return p;
}

cudaError_t launch_embed(const int64_t* tokens, const void* w, void* h, int64_t S, int Dm,
                         int64_t V, float scale, cudaStream_t stream) {
  const int vecs = Dm / 8, parts = (vecs + 127) / 128;
  const int64_t units = S * parts;
  launch_begin(kEmbedClass, stream);
  embed_kernel<<<static_cast<unsigned>((units + 7) / 8), 256, 0, stream>>>(
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
  const dim3 tiles(static_cast<unsigned>(p.tiles)), threads(kSortThreads);
  const int bins = 1 << p.bits;
  cudaError_t e = cudaSuccess;
  auto launch = [&](auto kernel, dim3 grid, dim3 block, bool early, auto... args) {
    if (e != cudaSuccess) return;
    launch_begin(kEmbedClass, stream);
    e = launch_after(kernel, grid, block, 0, stream, early, args...);
    launch_end(kEmbedClass, stream);
  };
  int in = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits, out = in ^ 1;
    const uint32_t *k = keys[in], *pl = places[in];
    if (pass == 0) {
      launch(sort_count_kernel<true>, tiles, threads, false, a, k, shift, bins);
    } else {
      launch(sort_count_kernel<false>, tiles, threads, true, a, k, shift, bins);
    }
    launch(sort_scan_kernel, dim3(1), dim3(1024), true, a.hist, p.tiles * bins);
    if (pass == 0)
      launch(sort_scatter_kernel<true>, tiles, threads, true, a, k, pl, keys[out], places[out],
             shift, p.bits);
    else
      launch(sort_scatter_kernel<false>, tiles, threads, true, a, k, pl, keys[out], places[out],
             shift, p.bits);
    in = out;
  }
  const int64_t zero = a.add ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
  const uint32_t *k = keys[in], *pl = places[in];
  launch(embed_sum_kernel, dim3(static_cast<unsigned>(p.chunks * p.slices + zero)),
         dim3(p.threads), true, a, k, pl);
  if (p.chunks > 1)
    launch(embed_join_kernel, dim3(static_cast<unsigned>(p.chunks * p.slices)), dim3(p.threads),
           true, a, k);
  return e;
}

}  // namespace upipe
