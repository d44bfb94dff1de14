// Token log probabilities out of the readout x = h w^T, with the entropy and the largest alternatives.
//
//   lse = M + ln z,  z = sum exp(x_j - M),  M = max x;   logp = (x_t - M) - ln z;
//   H = ln z - sum exp(x_j - M) (x_j - M) / z.
//
// The logits are made in groups of up to 128 columns, and never kept as a whole. Each group leaves, per
// row, its maximum, how often that occurs, and the sums of e = exp(x - max) and e (x - max) over the
// other columns. A probability near one leaves its mark in ln z alone, as z - 1; with the maximum's
// own ones counted apart that difference is a sum of small terms and keeps all its digits
// (ln z = ln count + ln(1 + rest / count)).
//
// The tensor cores' fp32 sums are truncated, not rounded: 4096 products that add up to 20 come out
// 8e-5 low. So an accumulator takes 512 products, and these sums are added up in registers, rounded to
// nearest, while the next ones run. Entropies of 512 rows, 4096 products a logit, against 64 bits:
// 1.7e-6 off with one accumulator for all, 1.8e-7 with 512 products, 0.9e-7 with 256, which takes 4 %
// longer where the tensor cores set the time. In short calls, where that costs nothing and a single
// logp near zero may be all that there is, an accumulator takes 64 products, and eight of them are
// added up before they are added to the others.
//
// Alternatives. The k largest logits lie in the k groups with the largest maxima (equal ones by index:
// an element outside has k elements before it). So logits are stored, and a row reads k groups of
// them: those not below the k-th largest maximum, which are few. Which of two logits is the larger is
// decided on sums that do not depend on how a kernel accumulates: kLogpMargin candidates behind the
// last one asked for are kept too, all are summed again in fp32 beside their length, which bounds the
// sum's error, and those that are nearer to each other than their bounds a third time, as a float
// and what it lost (every product of two bf16 is exact in fp32). Equal ones go by index.
//
// Up to 16 rows are bound by HBM: every row of w is read once. 128 rows of w are the M of an MMA, the
// few rows of h its N. More rows are bound by HBM up to about 250 and by the tensor cores beyond:
// 128 x 256 tiles of h and w, persistent blocks. Eight warps hold a tile's sums, 128 columns of a row
// each; the work on a finished tile runs beside the next one's first 512 products.
//
// Tiles have fewer columns than that where it fills the last round of blocks (LogpArgs::tile). It takes
// every SM's copies in flight to reach 7 TB/s: with whole tiles of 256, 48 tokens of 128256 columns are
// 3.3 rounds, of which the last 0.3 took as long as 0.7 of the others (174 us against 167 now, without
// alternatives); with one run of rows of w for each block, up to 16 tokens took 178 us, now 161.
#include <cfloat>

#include "internal.h"
#include "rope.cuh"

namespace upipe {
namespace {

constexpr int kClass = 18;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xffffffffu;

// ---- groups' sums -----------------------------------------------------------------------------

// Maximum, sum of e over the others, sum of e (x - max), how often the maximum occurs.
using Sums = float4;

__device__ __forceinline__ Sums no_sums() { return make_float4(-INFINITY, 0.f, 0.f, 0.f); }

// In memory the last word says how often the maximum occurs and which slices of 32 columns are stored.
__device__ __forceinline__ float mark(int count, uint32_t stored) {
  return __uint_as_float(static_cast<uint32_t>(count) | stored << 16);
}
__device__ __forceinline__ Sums read_sums(const float4& s) {
  return make_float4(s.x, s.y, s.z, static_cast<float>(__float_as_uint(s.w) & 0xffffu));
}

// Unsigned numbers in the order of the floats (-0 as +0); 0 is below all of them.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// s brought to the maximum m >= s.x, its own maximum among the others where m is larger.
__device__ __forceinline__ Sums rebase(const Sums& s, float m) {
  if (s.x == m) return s;
  if (s.x == -INFINITY) return make_float4(m, s.y, 0.f, 0.f);  // nothing, or NaN
  const float d = s.x - m, f = exp2f(d * kLog2e), n = s.y + s.w;
  return make_float4(m, f * n, f * fmaf(d, n, s.z), 0.f);
}

// ---- short calls ------------------------------------------------------------------------------

constexpr int kChunk = 1;  // stages of 64 products that one accumulator takes
constexpr int kShortThreads = 192;
constexpr int N = kLogpShortRows;
static_assert(N == 16, "an MMA's N, and the columns that load_columns loads");
constexpr int kAccs = 8;

struct ShortLayout {
  static constexpr int kA = 128 * 128, kB = N * 128, kStage = kA + kB;
  static constexpr int kTile = N * 128 * 4;  // the logits of a tile, [token][column]
  static constexpr int kStages = (224 * 1024 - kTile) / kStage;
  static constexpr int kX = kStages * kStage;
  static constexpr int kBar = kX + kTile;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccs + 1;
  static constexpr int kSlot = kBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kBytes = kSlot + 16 + 1024;
  static_assert(kBytes <= 227 * 1024, "a block's shared memory");
};

// 16 columns of this thread's row of an accumulator
__device__ __forceinline__ void load_columns(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int n = 0; n < 16; ++n) v[n] = __uint_as_float(r[n]);
}

// tm_w: boxes of a.tile rows, tm_h: of N (rows behind the last are zeros). A tile is a group.
__global__ void __launch_bounds__(kShortThreads, 1)
    logp_short_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_h, const LogpArgs a) {
  using L = ShortLayout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* acc_empty = acc_full + kAccs;
  uint64_t* drain = acc_empty + kAccs;
  float* tile = reinterpret_cast<float*>(smem + L::kX);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlot + 4);
  constexpr uint32_t kCols = kAccs * N;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = a.groups;
  const int nk = (a.Dm + 63) / 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  launch_dependents();

  auto wait = [&](uint64_t* br, uint32_t parity) -> bool {
    if (mbar_try_wait(br, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
      if (mbar_try_wait(br, parity)) return true;
      if ((n & 31) == 0) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(a.err, kErrWaitTimeout | 0x8000u);
          return false;
        }
      }
    }
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      int64_t fills = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        // (of 128 rows of A those behind the tile's last keep what was there: results not used)
        const uint32_t bytes = a.tile * 128u + L::kB;
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait(empty + s, ph ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * L::kStage;
          mbar_arrive_expect_tx(full + s, bytes);
          tma_load_3d(sa + L::kA, &tm_h, kb * 64, 0, 0, full + s);
          tma_load_3d(sa, &tm_w, kb * 64, t * a.tile, 0, full + s);
          ++fills;
          if (++s == L::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        // let the loads still in flight land before the block ends
        const int64_t first = fills > L::kStages ? fills - L::kStages : 0;
        for (int64_t f = first; f < fills; ++f)
          mbar_wait(full + (f % L::kStages), static_cast<uint32_t>((f / L::kStages) & 1),
                    100000000ull);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, N, false, false);
      const uint32_t s0 = smem_u32(smem);
      const uint64_t dA0 = kdesc0(s0), dB0 = kdesc0(s0 + L::kA);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 1;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        for (int kb = 0; kb < nk; ++kb) {
          const bool first = kb % kChunk == 0;
          if ((first && !wait(acc_empty + buf, acc_ph)) || !wait(full + s, ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tD = tmem + static_cast<uint32_t>(buf * N);
          const uint64_t dA = dA0 + s * (L::kStage >> 4), dB = dB0 + s * (L::kStage >> 4);
#pragma unroll
          for (int k16 = 0; k16 < 4; ++k16)
            umma_f16_ss(tD, dA + kstep(k16), dB + kstep(k16), idesc, !first || k16 > 0 ? 1u : 0u);
          umma_commit(empty + s);
          if (++s == L::kStages) {
            s = 0;
            ph ^= 1;
          }
          if (kb % kChunk == kChunk - 1 || kb == nk - 1) {
            umma_commit(acc_full + buf);
            if (++buf == kAccs) {
              buf = 0;
              acc_ph ^= 1;
            }
          }
        }
      }
      if (!ok) {
        umma_commit(drain);
        mbar_wait(drain, 0, 100000000ull);
      }
    }
  } else {
    // ---------------- sums: warps 2..5, a row of w each thread ----------------
    const int quarter = warp & 3;
    const int r = 32 * quarter + lane;
    const int chunks = (nk + kChunk - 1) / kChunk;
    int buf = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      float acc[N], few[N];  // sums of eight pieces at a time, and their sum: fewer roundings of large ones
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] = few[n] = 0.f;
      for (int c = 0; ok && c < chunks; ++c) {
        ok = __all_sync(kAll, wait(acc_full + buf, ph));
        if (!ok) break;
        tc_fence_after();
        float v[N];
        load_columns(tmem + (static_cast<uint32_t>(32 * quarter) << 16) +
                         static_cast<uint32_t>(buf * N), v);
#pragma unroll
        for (int n = 0; n < N; ++n) few[n] += v[n];
        if (c % 8 == 7 || c == chunks - 1) {
#pragma unroll
          for (int n = 0; n < N; ++n) {
            acc[n] += few[n];
            few[n] = 0.f;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + buf);
        if (++buf == kAccs) {
          buf = 0;
          ph ^= 1;
        }
      }
      // logits to [token][column], so that a warp takes a token's 128 at a time: sums over the
      // lanes once a token, not once a token and warp, and whole lines to memory
      asm volatile("bar.sync 1, 128;" ::: "memory");  // the tile before is done with
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n >= a.M) break;
        tile[n * 128 + r] = acc[n];
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const int left = group_width(a, t);
      const int64_t col = group_start(a, t) + 4 * lane;
#pragma unroll 2
      for (int n = quarter; n < a.M; n += 4) {
        float4 v = reinterpret_cast<const float4*>(tile + n * 128)[lane];
        if (4 * lane + 0 >= left) v.x = -INFINITY;
        if (4 * lane + 1 >= left) v.y = -INFINITY;
        if (4 * lane + 2 >= left) v.z = -INFINITY;
        if (4 * lane + 3 >= left) v.w = -INFINITY;
        const int64_t at = static_cast<int64_t>(n) * a.groups + t;
        if (a.logits && 4 * lane < left)
          *reinterpret_cast<float4*>(a.logits + at * kLogpWidth + 4 * lane) = v;
        const float x[4] = {v.x, v.y, v.z, v.w};
        if (a.target) {
          const int64_t k = a.target[n] - col;
          if (k >= 0 && k < 4 && 4 * lane + k < left)
            a.tlogit[n] = k == 0 ? x[0] : k == 1 ? x[1] : k == 2 ? x[2] : x[3];
        }
        float m = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        float sum = 0.f, sum1 = 0.f;
        int count = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = 4 * lane + k < left, top = x[k] == m;
          const float d = x[k] - m;
          const float e = top || !in ? 0.f : exp2f(d * kLog2e);  // NaN stays
          sum += e;
          if (in) sum1 = fmaf(e, fmaxf(d, -1000.f), sum1);
          count += __popc(__ballot_sync(kAll, top && in));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          sum += __shfl_xor_sync(kAll, sum, o);
          sum1 += __shfl_xor_sync(kAll, sum1, o);
        }
        if (lane == 0)
          a.part[at] = make_float4(m, sum, sum1, mark(count, 15u));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ---- longer calls -----------------------------------------------------------------------------

constexpr int kLongThreads = 320;
constexpr int kLongChunk = 8;  // stages of 64 products that one accumulator takes
constexpr int kLongGroup = 32;  // M tiles that are walked together: their rows of h stay in L2

struct LongLayout {
  static constexpr int kA = 128 * 128, kB = 256 * 128, kStage = kA + kB, kStages = 4;
  static constexpr int kBar = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kSlot = kBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kBytes = kSlot + 16 + 1024;
};

// Tile t: groups of kLongGroup M tiles, M first.
__device__ __forceinline__ void long_tile(int64_t t, int m_tiles, int n_tiles, int* mt, int* nt) {
  const int64_t per = static_cast<int64_t>(kLongGroup) * n_tiles;
  const int grp = static_cast<int>(div_fl(t, per));
  const int64_t rem = t - grp * per;
  const int wide = min(kLongGroup, m_tiles - grp * kLongGroup);
  *nt = static_cast<int>(div_fl(rem, wide));
  *mt = grp * kLongGroup + static_cast<int>(rem - static_cast<int64_t>(*nt) * wide);
}

// Sums, target and wanted logits of group g of one row: x, up to 128 columns from col0 to end.
// Logits are wanted for the row's `keep` largest alone. Slot g % keep of `best` holds the largest
// logit of every keep-th group so far, so the smallest of the slots is a bound below which no logit
// can be among them: a slice of 32 columns below it is not stored (of 4096 x 128256 logits 2 % are, with
// nine to keep, 6 % with 28; with all of them stored the call took 0.5 ms more). The bound only grows; an older
// one stores more, never less.
__device__ __forceinline__ void finish_row(const LogpArgs& a, int64_t row, int g, int col0, int end,
                                           uint32_t bound, float (&x)[128]) {
  if (col0 + 128 > end) {
    const int n = end - col0;
#pragma unroll
    for (int j = 0; j < 128; ++j)
      if (j >= n) x[j] = -INFINITY;
  }
  float top[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    top[s] = fmaxf(x[32 * s], x[32 * s + 1]);
#pragma unroll
    for (int j = 2; j < 32; j += 2) top[s] = fmax3(top[s], x[32 * s + j], x[32 * s + j + 1]);
  }
  const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  uint32_t stored = 0;
  if (a.logits) {
    atomicMax(a.best + static_cast<int64_t>(g % a.keep) * a.M + row, order_key(mx));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (col0 + 32 * s >= end || order_key(top[s]) < bound) continue;
      stored |= 1u << s;
      float4* dst = reinterpret_cast<float4*>(a.logits + (row * a.groups + g) * kLogpWidth + 32 * s);
#pragma unroll
      for (int v = 0; v < 8; ++v)
        dst[v] = make_float4(x[32 * s + 4 * v], x[32 * s + 4 * v + 1], x[32 * s + 4 * v + 2],
                             x[32 * s + 4 * v + 3]);
    }
  }
  float rest = 0.f, sum1 = 0.f;
  int count = 0;
#pragma unroll
  for (int j = 0; j < 128; ++j) {
    const float d = x[j] - mx;
    const float e = ex2_approx(d * kLog2e);
    const bool max = x[j] == mx;
    rest += max ? 0.f : e;
    count += max ? 1 : 0;
    sum1 = fmaf(e, fmaxf(d, -1000.f), sum1);  // d = 0 for the maximum; no 0 * inf for -inf
  }
  a.part[row * a.groups + g] = make_float4(mx, rest, sum1, mark(count, stored));
  if (a.target) {
    const int64_t k = a.target[row] - col0;
    if (k >= 0 && k < 128 && col0 + k < end) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < 128; ++j)  // (written as x[k], or as ?:, it would put x into local memory)
        asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, %3;\n\tselp.f32 %0, %1, %0, p;\n\t}"
            : "+f"(v)
            : "f"(x[j]), "r"(static_cast<int>(k)), "r"(j));
      a.tlogit[row] = v;
    }
  }
}

// Warp 0 loads, warp 1 multiplies, warps 2 .. 9 add up: warp w holds rows 32 (w % 4) .. + 31 of the tile
// and its first (w < 6) or second 128 columns. The two accumulators alternate between pieces of
// kLongChunk stages.
__global__ void __launch_bounds__(kLongThreads, 1)
    logp_long_kernel(const __grid_constant__ CUtensorMap tm_h,
                     const __grid_constant__ CUtensorMap tm_w, const LogpArgs a) {
  using L = LongLayout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlot + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tiles = (a.M + 127) / 128, n_tiles = logp_tiles(a);
  const int64_t tiles = static_cast<int64_t>(m_tiles) * n_tiles;
  const int nk = (a.Dm + 63) / 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](uint64_t* br, uint32_t parity) -> bool {
    if (mbar_try_wait(br, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
      if (mbar_try_wait(br, parity)) return true;
      if ((n & 31) == 0) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(a.err, kErrWaitTimeout | 0x8000u);
          return false;
        }
      }
    }
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tm_h);
      tma_prefetch_desc(&tm_w);
      int s = 0;
      uint32_t ph = 0;
      int64_t fills = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        int mt, nt;
        long_tile(t, m_tiles, n_tiles, &mt, &nt);
        for (int kb = 0; kb < nk; ++kb) {
          if (!wait(empty + s, ph ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * L::kStage;
          mbar_arrive_expect_tx(full + s, L::kA + a.tile * 128u);
          tma_load_3d(sa, &tm_h, kb * 64, mt * 128, 0, full + s);
          tma_load_3d(sa + L::kA, &tm_w, kb * 64, nt * a.tile, 0, full + s);
          ++fills;
          if (++s == L::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        // let the loads still in flight land before the block ends
        const int64_t first = fills > L::kStages ? fills - L::kStages : 0;
        for (int64_t f = first; f < fills; ++f)
          mbar_wait(full + (f % L::kStages), static_cast<uint32_t>((f / L::kStages) & 1),
                    100000000ull);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: the whole warp, converged; one lane's products go out ----------------
    const uint32_t idesc = idesc_bf16(128, (a.tile + 15) / 16 * 16, false, false);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t dA0 = kdesc0(s0), dB0 = kdesc0(s0 + L::kA);
    int s = 0, buf = 0;
    uint32_t ph = 0, acc_ph = 1;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      for (int kb = 0; kb < nk; ++kb) {
        const bool first = kb % kLongChunk == 0;
        ok = (!first || wait(acc_empty + buf, acc_ph)) && wait(full + s, ph);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tD = tmem + static_cast<uint32_t>(buf * 256);
        const uint64_t dA = dA0 + s * (L::kStage >> 4), dB = dB0 + s * (L::kStage >> 4);
#pragma unroll
        for (int k16 = 0; k16 < 4; ++k16)
          umma_f16_ss_warp(tD, dA + kstep(k16), dB + kstep(k16), idesc,
                           !first || k16 > 0 ? 1u : 0u);
        umma_commit_warp(empty + s);
        if (++s == L::kStages) {
          s = 0;
          ph ^= 1;
        }
        if (kb % kLongChunk == kLongChunk - 1 || kb == nk - 1) {
          umma_commit_warp(acc_full + buf);
          buf ^= 1;
          acc_ph ^= buf == 0;
        }
      }
    }
    if (!ok) {
      umma_commit_warp(drain);
      mbar_wait(drain, 0, 100000000ull);
    }
  } else {
    // ---------------- sums ----------------
    const int quarter = warp & 3, half = warp >= 6;
    const int chunks = (nk + kLongChunk - 1) / kLongChunk;
    const uint32_t mine = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 128u * half;
    int buf = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      int mt, nt;
      long_tile(t, m_tiles, n_tiles, &mt, &nt);
      const int64_t row = static_cast<int64_t>(mt) * 128 + 32 * quarter + lane;
      uint32_t bound = 0xffffffffu;
      if (a.logits && row < a.M) {
        // eight loads at a time: one after the other they would take longer than a piece of the tile
        for (int k0 = 0; k0 < a.keep; k0 += 8) {
          uint32_t v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int slot = k0 + k < a.keep ? k0 + k : k0;
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];"
                         : "=r"(v[k])
                         : "l"(a.best + static_cast<int64_t>(slot) * a.M + row));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) bound = min(bound, v[k]);
        }
      }
      float x[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) x[j] = 0.f;
      for (int c = 0; c < chunks; ++c) {
        ok = __all_sync(kAll, wait(acc_full + buf, ph));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float v[16];
          load_columns(mine + static_cast<uint32_t>(buf * 256 + 16 * q), v);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[16 * q + j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + buf);
        buf ^= 1;
        ph ^= buf == 0;
      }
      if (!ok || row >= a.M || 128 * half >= a.tile) continue;
      const int per = a.tile > kLogpWidth ? 2 : 1, g = nt * per + half;
      const int col0 = nt * a.tile + 128 * half;
      const int end = min((nt + 1) * a.tile, static_cast<int>(a.V));
      if (col0 < end)
        finish_row(a, row, g, col0, end, bound, x);
      else
        a.part[row * a.groups + g] = no_sums();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- rows' results ----------------------------------------------------------------------------

constexpr int kOwn = 4;  // groups that a thread keeps in registers

// The `want` (at most 32) items of [0, n) with the largest keys, equal ones by number, in any order, to
// list; returns how many there are. Items with a key below `least` (1 or more) do not count. A radix
// selection: the digits of the last one's key from the top, by counting, until the items with the
// digits so far are all wanted. The whole block calls.
template <int kThreads, typename Key>
__device__ int block_select(Key key, int n, int want, uint32_t least, int* list, uint32_t* counts) {
  __shared__ uint32_t prefix_s, need_s, exact_s, found_s;
  const int lane = threadIdx.x & 31;
  uint32_t prefix = 0, mask = 0, need = want;
  bool exact = false;
  for (int shift = 24; shift >= 0 && !exact; shift -= 8) {
    __syncthreads();
    for (int d = threadIdx.x; d < 256; d += kThreads) counts[d] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t k = key(i);
      if (k >= least && (k & mask) == prefix) atomicAdd(&counts[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // eight digits a lane, the largest first
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = counts[255 - 8 * lane - j];
      uint32_t up = sum;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint32_t o = __shfl_up_sync(kAll, up, m);
        if (lane >= m) up += o;
      }
      uint32_t above = up - sum;
      const uint32_t all = __shfl_sync(kAll, up, 31);
      if (all <= need) {  // (first digit) no more than are wanted
        if (lane == 0) {
          prefix_s = 0;
          need_s = all;
          exact_s = 1;
        }
      } else if (above < need && need <= up) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < need && need <= above + c[j]) {
            prefix_s = prefix | static_cast<uint32_t>(255 - 8 * lane - j) << shift;
            need_s = need - above;
            exact_s = need - above == c[j];
          }
          above += c[j];
        }
      }
      if (lane == 0) found_s = 0;
    }
    __syncthreads();
    prefix = prefix_s;
    need = need_s;
    exact = exact_s != 0;
    mask |= 255u << shift;
  }
  // exact: every key from the prefix on; else those above the prefix, which is a whole key now, and
  // the first `need` of its own
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t k = key(i);
    if (k >= least && (exact ? k >= prefix : k > prefix)) list[atomicAdd(&found_s, 1u)] = i;
  }
  __syncthreads();
  int found = static_cast<int>(found_s);
  if (!exact) {
    if (threadIdx.x < 32) {
      uint32_t taken = 0;
      for (int i0 = 0; taken < need; i0 += 32) {
        const bool is = i0 + lane < n && key(i0 + lane) == prefix;
        const uint32_t all = __ballot_sync(kAll, is);
        const uint32_t at = taken + __popc(all & ((1u << lane) - 1));
        if (is && at < need) list[found + at] = i0 + lane;
        taken += __popc(all);
      }
    }
    found += static_cast<int>(need);
    __syncthreads();
  }
  return found;
}

// Vectors k0, k0 + 256, .. of two rows of Dm bf16, asked for together: the rows come from anywhere in w.
constexpr int kAhead = 4;
struct Vectors {
  uint4 a[kAhead], b[kAhead];
  __device__ __forceinline__ void load(const __nv_bfloat16* h, const __nv_bfloat16* w, int k0, int Dm) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + 256 * j;
      a[j] = b[j] = make_uint4(0, 0, 0, 0);
      if (k < Dm) {
        b[j] = __ldg(reinterpret_cast<const uint4*>(w + k));
        a[j] = *reinterpret_cast<const uint4*>(h + k);
      }
    }
  }
};

// <h, w>, <h, h> and <w, w> in fp32, the part that falls to one warp of two (which: 0 or 1; turns of
// 256 kAhead features). A term of the first is rounded 4 times in its vector, once for each of the
// lane's vectors (kAhead a turn) and 7 times across lanes and warps.
__device__ __forceinline__ float3 dot_near(const __nv_bfloat16* h, const __nv_bfloat16* w, int Dm,
                                           int which) {
  uint64_t hw = 0, hh = 0, ww = 0;
  for (int k0 = which * 256 * kAhead + (threadIdx.x & 31) * 8; k0 < Dm; k0 += 2 * 256 * kAhead) {
    Vectors v;
    v.load(h, w, k0, Dm);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t x[4] = {v.a[j].x, v.a[j].y, v.a[j].z, v.a[j].w};
      const uint32_t y[4] = {v.b[j].x, v.b[j].y, v.b[j].z, v.b[j].w};
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t p = f2_pack_u(x[i] << 16, x[i] & 0xffff0000u);
        const uint64_t q = f2_pack_u(y[i] << 16, y[i] & 0xffff0000u);
        sum = ffma2(p, q, sum);
        hh = ffma2(p, p, hh);
        ww = ffma2(q, q, ww);
      }
      hw = fadd2(hw, sum);
    }
  }
  float3 r;
  float lo, hi;
  f2_unpack(hw, lo, hi);
  r.x = lo + hi;
  f2_unpack(hh, lo, hi);
  r.y = lo + hi;
  f2_unpack(ww, lo, hi);
  r.z = lo + hi;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    r.x += __shfl_xor_sync(kAll, r.x, o);
    r.y += __shfl_xor_sync(kAll, r.y, o);
    r.z += __shfl_xor_sync(kAll, r.z, o);
  }
  return r;
}

// The same part of <h, w> with an error near 2^-45 of the terms: each lane keeps its sums and the sums of
// what each addition lost (Knuth's error-free transformation of a sum).
__device__ __forceinline__ double dot_exact(const __nv_bfloat16* h, const __nv_bfloat16* w, int Dm,
                                            int which) {
  float s[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};
  for (int k0 = which * 256 * kAhead + (threadIdx.x & 31) * 8; k0 < Dm; k0 += 2 * 256 * kAhead) {
    Vectors v;
    v.load(h, w, k0, Dm);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      float x[8], y[8];
      unpack_bf16x8(v.a[j], x);
      unpack_bf16x8(v.b[j], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float& u = s[i & 1];
        const float p = __fmul_rn(x[i], y[i]);
        const float t = __fadd_rn(u, p);
        const float z = __fadd_rn(t, -u);
        lost[i & 1] = __fadd_rn(lost[i & 1],
                                __fadd_rn(__fadd_rn(u, -__fadd_rn(t, -z)), __fadd_rn(p, -z)));
        u = t;
      }
    }
  }
  double d = (static_cast<double>(s[0]) + static_cast<double>(s[1])) +
             (static_cast<double>(lost[0]) + static_cast<double>(lost[1]));
#pragma unroll
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(kAll, d, o);
  return d;
}

constexpr int kFew = 128;  // logits of a row that are ranked one against the other

// One block per row. smem: `keep` groups of `width` logits.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) logp_pick_kernel(const LogpArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ float picked[];
  __shared__ float red[kWarps][3];
  __shared__ float row_ln;
  __shared__ uint32_t counts[256];
  __shared__ int list[32], grp[32], cand[32];
  __shared__ uint32_t grp_least, last_key, grp_mark[32];
  __shared__ uint32_t segment[32];
  __shared__ float cand_x[32];
  __shared__ float3 cand_n[32][2];
  __shared__ double cand_y[32], cand_e[32][2];
  __shared__ uint32_t near_mask;
  __shared__ uint32_t few_key[kFew];
  __shared__ uint32_t few_mark[kFew];
  __shared__ int few_col[kFew], few_rank[kFew], few_n;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  const float4* part = a.part + row * a.groups;

  // a thread's groups, and the largest of each 32nd group
  float4 own[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int g = threadIdx.x + k * kThreads;
    own[k] = g < a.groups ? part[g] : no_sums();
  }
  if (threadIdx.x < 32) segment[threadIdx.x] = 0;
  if (threadIdx.x == 0) few_n = 0;
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) m = fmaxf(m, own[k].x);
  for (int g = threadIdx.x + kOwn * kThreads; g < a.groups; g += kThreads) m = fmaxf(m, part[g].x);
  __syncthreads();
  if (threadIdx.x < a.groups) atomicMax(&segment[lane], order_key(m));
  __syncthreads();
  uint32_t top_key = segment[lane];
  if (warp == 0) {
    // as many groups as are kept have a maximum from the keep-th largest of these on
    int rank = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const uint32_t u = __shfl_sync(kAll, top_key, k);
      rank += u > top_key || (u == top_key && k < lane);
    }
    static_assert(kLogpMaxTop + kLogpMargin <= 32, "the kept ones, a lane each");
    if (rank == a.keep - 1) grp_least = max(top_key, 1u);
  }
  top_key = __reduce_max_sync(kAll, top_key);
  m = __uint_as_float(top_key & 0x80000000u ? top_key ^ 0x80000000u : ~top_key);
  float rest = 0.f, sum1 = 0.f, count = 0.f;
  auto add = [&](const Sums& s) {
    const Sums u = rebase(s, m);
    rest += u.y;
    sum1 += u.z;
    count += u.w;
  };
#pragma unroll
  for (int k = 0; k < kOwn; ++k) add(read_sums(own[k]));
  for (int g = threadIdx.x + kOwn * kThreads; g < a.groups; g += kThreads) add(read_sums(part[g]));
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    rest += __shfl_xor_sync(kAll, rest, o);
    sum1 += __shfl_xor_sync(kAll, sum1, o);
    count += __shfl_xor_sync(kAll, count, o);
  }
  if (lane == 0) {
    red[warp][0] = rest;
    red[warp][1] = sum1;
    red[warp][2] = count;
  }
  __syncthreads();
  if (warp == kWarps - 1) {  // (the others go on: ln is wanted at the end)
    rest = lane < kWarps ? red[lane][0] : 0.f;
    sum1 = lane < kWarps ? red[lane][1] : 0.f;
    count = lane < kWarps ? red[lane][2] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      rest += __shfl_xor_sync(kAll, rest, o);
      sum1 += __shfl_xor_sync(kAll, sum1, o);
      count += __shfl_xor_sync(kAll, count, o);
    }
    // a row with a logit of NaN or +inf, or without a finite one, has no probabilities
    float ln = logf(count) + log1pf(rest / count);
    if (!(fabsf(m) <= FLT_MAX)) ln = __int_as_float(0x7fc00000);
    if (lane == 0) {
      if (a.lse) a.lse[row] = m + ln;
      if (a.entropy) a.entropy[row] = ln - sum1 / (count + rest);
      if (a.logp) {
        const int64_t t = a.target[row];
        a.logp[row] = t < 0 ? 0.f : t < a.V ? (a.tlogit[row] - m) - ln : __int_as_float(0x7fc00000);
      }
      row_ln = ln;
    }
  }
  if (!a.top) return;
  float* out_v = a.top_logp + row * a.top;
  int64_t* out_i = a.top_index + row * a.top;

  // the groups with the largest maxima (one behind the last column has none), by number
  auto offer = [&](int g, const float4& p) {
    const uint32_t key = order_key(p.x);
    if (g >= a.groups || key < grp_least || group_width(a, g) <= 0) return;
    const int at = atomicAdd(&few_n, 1);
    if (at >= kFew) return;
    few_key[at] = key;
    few_col[at] = g;
    few_mark[at] = __float_as_uint(p.w);
  };
#pragma unroll
  for (int k = 0; k < kOwn; ++k) offer(threadIdx.x + k * kThreads, own[k]);
  for (int g = threadIdx.x + kOwn * kThreads; g < a.groups; g += kThreads) offer(g, part[g]);
  __syncthreads();
  const float ln = row_ln;
  if (!(fabsf(ln) <= FLT_MAX)) {
    for (int k = threadIdx.x; k < a.top; k += kThreads) {
      out_v[k] = __int_as_float(0x7fc00000);
      out_i[k] = -1;
    }
    return;
  }
  int groups = few_n;
  if (groups <= kFew) {
    // of these, each one's place among the wanted ones by number
    for (int i = threadIdx.x; i < groups; i += kThreads) {
      const uint32_t key = few_key[i];
      const int g = few_col[i];
      int rank = 0;
      for (int k = 0; k < groups; ++k) rank += few_key[k] > key || (few_key[k] == key && few_col[k] < g);
      few_rank[i] = rank;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < groups; i += kThreads) {
      if (few_rank[i] >= a.keep) continue;
      int at = 0;
      for (int k = 0; k < groups; ++k) at += few_rank[k] < a.keep && few_col[k] < few_col[i];
      grp[at] = few_col[i];
      grp_mark[at] = few_mark[i];
      if (few_rank[i] == a.keep - 1) last_key = few_key[i];
    }
    groups = min(groups, a.keep);
  } else {
    auto group_key = [&](int g) { return group_width(a, g) > 0 ? order_key(part[g].x) : 0u; };
    groups = block_select<kThreads>(group_key, a.groups, a.keep, 1u, list, counts);
    if (threadIdx.x < 32) {
      const int mine = lane < groups ? list[lane] : 0x7fffffff;
      int rank = 0;
      for (int k = 0; k < groups; ++k) rank += list[k] < mine;
      uint32_t least = 0xffffffffu;
      if (lane < groups) {
        grp[rank] = mine;
        grp_mark[rank] = __float_as_uint(part[mine].w);
        least = order_key(part[mine].x);
      }
      least = __reduce_min_sync(kAll, least);
      if (lane == 0) last_key = least;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) few_n = 0;
  // with as many groups as are kept, their maxima are as many logits: none below counts
  const uint32_t least = groups == a.keep ? last_key : 1u;
  __syncthreads();
  // their logits from the smallest of these maxima on; columns that were not stored are below it
  const float* x = a.logits + row * a.groups * kLogpWidth;
  for (int k = warp; k < groups; k += kWarps) {
    const int64_t c0 = static_cast<int64_t>(grp[k]) * kLogpWidth;
    const int n = group_width(a, grp[k]);
    const uint32_t stored = grp_mark[k] >> 16;
    for (int c = lane; c < kLogpWidth; c += 32) {
      const float v = c < n && (stored >> (c >> 5) & 1) ? x[c0 + c] : NAN;
      picked[k * kLogpWidth + c] = v;
      const uint32_t key = order_key(v);
      if (v == v && key >= least) {
        const int at = atomicAdd(&few_n, 1);
        if (at < kFew) {
          few_key[at] = key;
          few_col[at] = k * kLogpWidth + c;  // in the order of the columns
        }
      }
    }
  }
  __syncthreads();
  int found = few_n;
  if (found <= kFew) {
    for (int i = threadIdx.x; i < few_n; i += kThreads) {
      const uint32_t key = few_key[i];
      const int at = few_col[i];
      int rank = 0;
      for (int k = 0; k < few_n; ++k) rank += few_key[k] > key || (few_key[k] == key && few_col[k] < at);
      if (rank < a.keep) list[rank] = at;
    }
    found = min(found, a.keep);
    __syncthreads();
  } else {
    found = block_select<kThreads>(
        [&](int i) {
          const float v = picked[i];
          return v == v ? order_key(v) : 0u;
        },
        groups * kLogpWidth, a.keep, least, list, counts);
  }
  if (threadIdx.x < 32 && static_cast<int>(threadIdx.x) < found) {
    const int i = list[threadIdx.x], k = i / kLogpWidth;
    cand[threadIdx.x] = static_cast<int>(group_start(a, grp[k])) + i - k * kLogpWidth;
    cand_x[threadIdx.x] = picked[i];
  }
  __syncthreads();
  const __nv_bfloat16* h = a.h + row * a.Dm;
  for (int k = warp; k < 2 * found; k += kWarps) {
    const float3 n = dot_near(h, a.w + static_cast<int64_t>(cand[k >> 1]) * a.Dm, a.Dm, k & 1);
    if (lane == 0) cand_n[k >> 1][k & 1] = n;
  }
  __syncthreads();
  if (warp == 0) {
    float v = 0.f, bound = 0.f;
    if (lane < found) {
      const float3 n = cand_n[lane][0], o = cand_n[lane][1];
      v = n.x + o.x;
      // each rounding loses at most 2^-24 of the terms' magnitudes, whose sum is at most the product of
      // the lengths (themselves good to 1 % for any Dm)
      bound = (kAhead * ((a.Dm + 512 * kAhead - 1) / (512 * kAhead)) + 12) * 0x1p-24f * 1.01f * sqrtf(n.y + o.y) *
              sqrtf(n.z + o.z);
    }
    bool near = false;
    for (int k = 0; k < found; ++k) {
      const float u = __shfl_sync(kAll, v, k), e = __shfl_sync(kAll, bound, k);
      // (what is not finite is near everything)
      if (k != lane && !(fabsf(u - v) > e + bound)) near = true;
    }
    const uint32_t all = __ballot_sync(kAll, near && lane < found);
    if (lane == 0) near_mask = all;
    cand_y[lane] = v;
  }
  __syncthreads();
  const uint32_t again = near_mask;
  if (again) {
    const int n = __popc(again);
    for (int k = warp; k < 2 * n; k += kWarps) {
      const int c = __fns(again, 0, (k >> 1) + 1);
      const double y = dot_exact(h, a.w + static_cast<int64_t>(cand[c]) * a.Dm, a.Dm, k & 1);
      if (lane == 0) cand_e[c][k & 1] = y;
    }
    __syncthreads();
    if (threadIdx.x < 32 && (again >> lane & 1)) {
      const double y = cand_e[lane][0] + cand_e[lane][1];
      // where infinities or an overflow leave no sum, the order is that of the logits
      cand_y[lane] = fabs(y) <= DBL_MAX ? y : static_cast<double>(cand_x[lane]);
    }
    __syncwarp();
  }
  if (threadIdx.x >= 32) return;
  if (lane >= found && lane < a.top) {  // fewer columns than asked for
    out_v[lane] = -INFINITY;
    out_i[lane] = -1;
  }
  if (lane >= found) return;
  const double y = cand_y[lane];
  const int me = cand[lane];
  int rank = 0;
  for (int k = 0; k < found; ++k)
    if (cand_y[k] > y || (cand_y[k] == y && cand[k] < me)) ++rank;
  if (rank < a.top) {
    out_v[rank] = (cand_x[lane] - m) - ln;
    out_i[rank] = me;
  }
}

}  // namespace

cudaError_t launch_logp_short(const CUtensorMap& tw, const CUtensorMap& th, const LogpArgs& a,
                              cudaStream_t stream) {
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&logp_short_kernel),
                                   ShortLayout::kBytes);
  if (e != cudaSuccess) return e;
  launch_begin(kClass, stream);
  const int blocks = a.groups < kLogpBlocks ? a.groups : kLogpBlocks;
  logp_short_kernel<<<blocks, kShortThreads, ShortLayout::kBytes, stream>>>(tw, th, a);
  e = cudaGetLastError();
  launch_end(kClass, stream);
  return e;
}

cudaError_t launch_logp_long(const CUtensorMap& th, const CUtensorMap& tw, const LogpArgs& a, int sms,
                             cudaStream_t stream) {
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&logp_long_kernel),
                                   LongLayout::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((a.M + 127) / 128) * logp_tiles(a);
  launch_begin(kClass, stream);
  logp_long_kernel<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kLongThreads,
                     LongLayout::kBytes, stream>>>(th, tw, a);
  e = cudaGetLastError();
  launch_end(kClass, stream);
  return e;
}

cudaError_t launch_logp_pick(const LogpArgs& a, cudaStream_t stream) {
  const size_t smem = a.top ? static_cast<size_t>(a.keep) * kLogpWidth * 4 : 0;
  const dim3 grid(static_cast<unsigned>(a.M));
  launch_begin(kClass, stream);
  // Few rows: a whole SM's warps each, for the latency of a row. More: what hides it is other rows.
  // Only a single block may start early: several would all go to the first SM that is free.
  const cudaError_t e =
      a.M <= 152 ? launch_after(logp_pick_kernel<1024>, grid, dim3(1024), smem, stream, a.M == 1, a)
                 : launch_after(logp_pick_kernel<256>, grid, dim3(256), smem, stream, false, a);
  launch_end(kClass, stream);
  return e;
}

}  // namespace upipe
