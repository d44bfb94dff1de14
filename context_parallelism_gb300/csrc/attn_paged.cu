// Attention of a batch's new tokens over a paged key/value cache: the prefix that the whole batch
// shares, computed once for all its rows, and each sequence's own pages.
//
// Row (sequence b, new token i of n, q-head h) sees the prefix's keys 0..P-1 and its own keys
// 0..len_b - n + i. Per kv-head, an item is a tile of rows (the G q-heads of consecutive tokens;
// of all sequences for the prefix, of one for its own pages) against one range of keys:
//   s = scale <q, k>,  m = max s,  p = exp2(s - m) (log2 units),  O~ = sum p v,  l = sum p,
// one pass with the running maximum and sum. An item's (m, l, O~) is one part of its rows; the
// parts of a row are joined by
//   M = max m_p,  o = sum 2^(m_p - M) O~_p / sum 2^(m_p - M) l_p,  lse = ln 2 (M + log2 l).
// P is rounded to bf16 for the P V product. Two sums are kept: that of the rounded weights
// divides O~ (numerator and denominator agree), that of the fp32 weights gives lse.
//
// Bound: HBM (each key and value is read once per row tile; 4 bytes per key feature carry
// 4 x rows FLOP). The matrix instruction is mma.sync m16n8k16: a decode step has G to 16 rows a
// kv-head, which a 128-row tcgen05 tile would fill to an eighth at most.
//
// Block: one producer warp (TMA boxes of page rows into a ring of 64-key stages) and four
// consumer warps. Row tiles of 16 split each stage's keys over the four warps (16 each), which
// join their statistics at the end; row tiles of 64 give each warp 16 rows and all keys.
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"

namespace upipe {
namespace {

constexpr int kKeys = 64;     // keys per stage
constexpr int kThreads = 160;  // 4 consumer warps + 1 producer warp

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int x, int y,
                                            int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int MT>
struct PLayout {
  static constexpr int kStage = 2 * kKeys * D * 2;  // K then V
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kMl = kStages * kStage;      // 16-row tiles: 4 warps x 16 rows float4
  static constexpr int kBar = kMl + 4 * 16 * 16;
  static constexpr int kAbort = kBar + (2 * kStages + 2) * 8;
  static constexpr int kBytes = kAbort + 16 + 1024;
};

// Rows [row0, row0 + n_rows) of an item in (token, head-of-group) order, and its key range.
struct Item {
  int kvh;
  int part;
  int b;             // own sequence (-1: the prefix)
  int64_t tok0;      // first token (row of q) of the segment
  int64_t n_tok;     // tokens of the segment
  int64_t k_lo, k_hi;
  int64_t own_before;  // own keys that the first token sees less one (causal limit), own items
  const int32_t* pages;
  int64_t n_table;
};

__device__ __forceinline__ int64_t row_limit(const Item& it, int64_t i) {
  return it.b < 0 ? it.k_hi : min(it.k_hi, it.own_before + i + 1);
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using L = PLayout<D, MT>;
  constexpr int KW = MT == 16 ? 16 : 64;  // keys of a stage that one warp works on
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* meet = empty + L::kStages;  // the four consumer warps among themselves
  uint64_t* joined = meet + 1;          // 16-row tiles: the stages' memory is free again
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4);
    }
    mbar_init(meet, 4);
    mbar_init(joined, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  // ---- which item ------------------------------------------------------------------------
  Item it;
  int tile, n_tiles;
  {
    int64_t x = blockIdx.x;
    const int64_t n_p =
        a.splits_x ? 0 : static_cast<int64_t>(a.splits_p) * a.tiles_p * a.Hkv;
    int split, splits;
    if (x < n_p) {
      it.kvh = static_cast<int>(x % a.Hkv);
      x /= a.Hkv;
      tile = static_cast<int>(x % a.tiles_p);
      split = static_cast<int>(x / a.tiles_p);
      n_tiles = a.tiles_p;
      splits = a.splits_p;
      it.part = split;
      it.b = -1;
      it.tok0 = 0;
      it.n_tok = a.rows;
      if (a.cu) it.n_tok = min(a.rows, max(static_cast<int64_t>(a.cu[a.B]), int64_t(0)));
      it.k_lo = 0;
      it.k_hi = a.prefix;
      it.own_before = 0;
      it.pages = a.ptable;
      it.n_table = (a.prefix + a.page_size - 1) / a.page_size;
    } else {
      x -= n_p;
      it.kvh = static_cast<int>(x % a.Hkv);
      x /= a.Hkv;
      tile = static_cast<int>(x % a.tiles_o);
      x /= a.tiles_o;
      split = static_cast<int>(x % a.splits_o);
      it.b = static_cast<int>(x / a.splits_o);
      n_tiles = a.tiles_o;
      splits = a.splits_o;
      it.part = a.splits_p + split;
      if (a.cu) {
        const int64_t c0 = a.cu[it.b], c1 = a.cu[it.b + 1];
        it.tok0 = min(max(c0, int64_t(0)), a.rows);
        it.n_tok = max(min(c1, a.rows) - it.tok0, int64_t(0));
      } else {
        it.tok0 = it.b * a.T;
        it.n_tok = a.T;
      }
      const int64_t cap = a.max_pages * a.page_size;
      int64_t len = a.seq_len[it.b];
      if (len > cap && threadIdx.x == 0) atomicOr(a.err, kErrBadPage);
      len = min(max(len, int64_t(0)), cap);
      it.k_lo = 0;
      it.k_hi = len;
      it.own_before = len - it.n_tok;
      it.pages = a.table + it.b * a.table_stride;
      it.n_table = a.max_pages;
    }
    // this split's share of the 64-key tiles, at least four of them
    const int64_t nt = (it.k_hi + kKeys - 1) / kKeys;
    const int64_t share = max((nt + splits - 1) / splits, int64_t(4));
    it.k_lo = min(it.k_hi, split * share * kKeys);
    it.k_hi = min(it.k_hi, (split + 1) * share * kKeys);
  }
  const int n_kt = static_cast<int>((it.k_hi - it.k_lo + kKeys - 1) / kKeys);
  const int64_t n_rows = it.n_tok * a.G;

  auto wait = [&](uint64_t* br, uint32_t parity) -> bool {
    if (mbar_try_wait(br, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
      if (mbar_try_wait(br, parity)) return true;
      if ((n & 31) == 0) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(a.err, kErrWaitTimeout | 0x10000u);
          return false;
        }
      }
    }
  };

  if (warp == 4) {
    // ---------------- producer: lane x loads box x of each stage ----------------
    const int bx = a.box_rows;  // divides page_size and 64
    const int boxes = kKeys / bx * (D / 64);
    uint32_t n_it = 0;
    bool ok = true;
    uint32_t n_rt = 0;
    for (int64_t rt = tile; ok && rt * MT < n_rows; rt += n_tiles, ++n_rt) {
      if (MT == 16 && n_rt > 0)
        ok = __all_sync(0xffffffffu, wait(joined, (n_rt - 1) & 1));
      for (int j = 0; ok && j < n_kt; ++j, ++n_it) {
        const int s = static_cast<int>(n_it % L::kStages);
        const uint32_t ph = n_it / L::kStages;
        if (ph > 0) ok = __all_sync(0xffffffffu, wait(empty + s, (ph - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + s, L::kStage);
        __syncwarp();
        const uint32_t base = smem_u32(smem) + s * L::kStage;
        const int64_t k0 = it.k_lo + static_cast<int64_t>(j) * kKeys;
        for (int x = lane; x < boxes; x += 32) {
          const int r = x / (D / 64) * bx, half = x % (D / 64);
          const int64_t key = k0 + r;
          // A box past the keys, or of a page that does not exist, lies outside the tensor map
          // and reads as zeros; nothing outside the caches is touched.
          int page = -1, slot = 0;
          if (key < it.k_hi) {
            const int64_t pg = key / a.page_size;
            page = pg < it.n_table ? it.pages[pg] : -1;
            slot = static_cast<int>(key - pg * a.page_size);
            if (page < 0 || page >= a.n_pages) {
              page = -1;
              atomicOr(a.err, kErrBadPage);
            }
          }
          const uint32_t dst = base + half * (kKeys * 128) + r * 128;
          tma_load_4d(dst, &tm_k, half * 64, slot, it.kvh, page, full + s);
          tma_load_4d(dst + kKeys * D * 2, &tm_v, half * 64, slot, it.kvh, page, full + s);
        }
      }
    }
    if (!ok) {  // copies in flight land before the block's shared memory goes
      for (uint32_t j = (n_it >= L::kStages ? n_it - L::kStages : 0); j < n_it; ++j)
        mbar_wait(full + j % L::kStages, (j / L::kStages) & 1, 100000000ull);
    }
  } else {
    // ---------------- consumers ----------------
    const int kw0 = MT == 16 ? warp * 16 : 0;
    const int r_lo = lane >> 2;
    const uint32_t sm0 = smem_u32(smem);
    const bool sole = a.splits_p + a.splits_o == 1;
    uint32_t n_it = 0, n_meet = 0;
    bool ok = true;
    // Every consumer warp has come here, and sees what the others wrote; false on expiry.
    auto meet_all = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      return __all_sync(0xffffffffu, wait(meet, n_meet++ & 1));
    };
    for (int64_t rt = tile; ok && rt * MT < n_rows; rt += n_tiles) {
      // this thread's two rows: token, head and key limit
      int64_t tok[2];
      int head[2];
      int64_t lim[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t r = rt * MT + (MT == 16 ? 0 : warp * 16) + r_lo + 8 * e;
        const int64_t i = r / a.G;
        head[e] = it.kvh * a.G + static_cast<int>(r - i * a.G);
        tok[e] = r < n_rows ? it.tok0 + i : -1;
        lim[e] = r < n_rows ? row_limit(it, i) : it.k_lo;
      }
      uint32_t qf[D / 16][4];
      {
        const __nv_bfloat16* qp[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t t = tok[e];
          const int64_t bb = a.cu ? 0 : t / a.T, ii = a.cu ? t : t - bb * a.T;
          qp[e] = t < 0 ? nullptr : a.q + bb * a.q_b + ii * a.q_s + head[e] * a.q_h + (lane & 3) * 2;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            qf[k][e] = qp[e & 1] ? *reinterpret_cast<const uint32_t*>(qp[e & 1] + k * 16 + (e >> 1) * 8)
                                 : 0u;
      }
      float o[D / 8][4];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, lb[2] = {0.f, 0.f}, lf[2] = {0.f, 0.f};

      for (int j = 0; j < n_kt; ++j, ++n_it) {
        const int s = static_cast<int>(n_it % L::kStages);
        ok = __all_sync(0xffffffffu, wait(full + s, (n_it / L::kStages) & 1));
        if (!ok) break;
        const uint32_t sk = sm0 + s * L::kStage, sv = sk + kKeys * D * 2;
        const int64_t k0 = it.k_lo + static_cast<int64_t>(j) * kKeys;
        // Values past the range's last key (slots of its last page that no token fills) may be
        // anything, infinities and NaN among them, and 0 * inf is not 0: they are cleared.
        if (k0 + kKeys > it.k_hi) {
          const int valid = static_cast<int>(it.k_hi - k0);
          for (int x = lane; x < 16 * (D / 8); x += 32) {
            const int r = warp * 16 + x / (D / 8), ch = x % (D / 8);
            if (r >= valid)
              st_shared_v4(sv + (ch >> 3) * (kKeys * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                           0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // before TMA may fill the stage again
          if (MT == 16) __syncwarp();
          else ok = meet_all();
          if (!ok) break;
        }
        float sc[KW / 8][4];
#pragma unroll
        for (int n = 0; n < KW / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int ch = (k & 3) * 2 + ((lane >> 3) & 1);
#pragma unroll
          for (int kg = 0; kg < KW / 16; ++kg) {
            const int r = kw0 + kg * 16 + ((lane >> 4) << 3) + (lane & 7);
            uint32_t kb[4];
            ldsm4(kb, sk + (k >> 2) * (kKeys * 128) + r * 128 + ((ch ^ (r & 7)) << 4));
            mma16816(sc[2 * kg], qf[k], kb[0], kb[1]);
            mma16816(sc[2 * kg + 1], qf[k], kb[2], kb[3]);
          }
        }
        // scale, mask, running maximum
        const int64_t kb0 = k0 + kw0 + (lane & 3) * 2;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < KW / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool seen = kb0 + n * 8 + (e & 1) < lim[e >> 1];
            sc[n][e] = seen ? sc[n][e] * a.scale_log2 : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
          }
        float al[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          base[e] = mx[e] == -INFINITY ? 0.f : mx[e];
          al[e] = ex2_approx(m[e] - base[e]);
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= al[e >> 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            lb[e] *= al[e];
            lf[e] *= al[e];
            m[e] = mx[e];
          }
        }
        // weights, rounded to bf16 once for the product
        uint32_t pf[KW / 16][4];
#pragma unroll
        for (int n = 0; n < KW / 8; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = ex2_approx(sc[n][2 * e] - base[e]);
            const float p1 = ex2_approx(sc[n][2 * e + 1] - base[e]);
            const uint32_t p = pack_bf16(p0, p1);
            lf[e] += p0 + p1;
            float b0 = lb[e], b1 = 0.f;
            add_bf16x2(b0, b1, p);
            lb[e] = b0 + b1;
            pf[n >> 1][(n & 1) * 2 + e] = p;
          }
        }
#pragma unroll
        for (int kg = 0; kg < KW / 16; ++kg)
#pragma unroll
          for (int dp = 0; dp < D / 16; ++dp) {
            const int r = kw0 + kg * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
            const int ch = (dp & 3) * 2 + (lane >> 4);
            uint32_t vb[4];
            ldsm4_t(vb, sv + (dp >> 2) * (kKeys * 128) + r * 128 + ((ch ^ (r & 7)) << 4));
            mma16816(o[2 * dp], pf[kg], vb[0], vb[1]);
            mma16816(o[2 * dp + 1], pf[kg], vb[2], vb[3]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + s);
      }
      if (!ok) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lb[e] += __shfl_xor_sync(0xffffffffu, lb[e], 1);
        lb[e] += __shfl_xor_sync(0xffffffffu, lb[e], 2);
        lf[e] += __shfl_xor_sync(0xffffffffu, lf[e], 1);
        lf[e] += __shfl_xor_sync(0xffffffffu, lf[e], 2);
      }
      if (MT == 16) {
        // join the four warps' key shares: statistics first, then the numerators
        float4* ml = reinterpret_cast<float4*>(smem + L::kMl);
        if ((lane & 3) == 0)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            ml[warp * 16 + r_lo + 8 * e] = make_float4(m[e], lb[e], lf[e], 0.f);
        ok = meet_all();
        if (!ok) break;
        float w[2];
        float4 all[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r_lo + 8 * e;
          float M = -INFINITY;
#pragma unroll
          for (int u = 0; u < 4; ++u) M = fmaxf(M, ml[u * 16 + r].x);
          const float bs = M == -INFINITY ? 0.f : M;
          all[e] = make_float4(M, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 v = ml[u * 16 + r];
            const float f = ex2_approx(v.x - bs);
            all[e].y += f * v.y;
            all[e].z += f * v.z;
          }
          w[e] = ex2_approx(m[e] - bs);
        }
        // Numerators go through the stages' memory: every copy of this row tile has landed and
        // been read. Row r of warp u at ((u * 16 + r) * (D + 4)) floats.
        float* ob = reinterpret_cast<float*>(smem);
        constexpr int kPitch = D + 4;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(ob + (warp * 16 + r_lo + 8 * e) * kPitch + n * 8 +
                                       (lane & 3) * 2) =
                make_float2(o[n][2 * e] * w[e], o[n][2 * e + 1] * w[e]);
        ok = meet_all();
        if (!ok) break;
        // warp u finishes rows 4u .. 4u+3, a lane D/32 features each
        for (int q = 0; q < 4; ++q) {
          const int r = warp * 4 + q;
          const int64_t row = rt * 16 + r;
          if (row >= n_rows) break;
          float v[D / 32];
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            const int d = lane * (D / 32) + x;
            v[x] = (ob[r * kPitch + d] + ob[(16 + r) * kPitch + d]) +
                   (ob[(32 + r) * kPitch + d] + ob[(48 + r) * kPitch + d]);
          }
          const int src = (r & 7) * 4;
          float4 st;
          st.x = __shfl_sync(0xffffffffu, r < 8 ? all[0].x : all[1].x, src);
          st.y = __shfl_sync(0xffffffffu, r < 8 ? all[0].y : all[1].y, src);
          st.z = __shfl_sync(0xffffffffu, r < 8 ? all[0].z : all[1].z, src);
          const int64_t i = row / a.G;
          const int h = it.kvh * a.G + static_cast<int>(row - i * a.G);
          const int64_t t = it.tok0 + i;
          if (sole) {
            const int64_t bb = a.cu ? 0 : t / a.T, ii = a.cu ? t : t - bb * a.T;
            const float inv = st.y == 0.f ? 0.f : 1.f / st.y;
            __nv_bfloat16* op = a.o + bb * a.o_b + ii * a.o_s + h * a.o_h + lane * (D / 32);
#pragma unroll
            for (int x = 0; x < D / 32; x += 2)
              *reinterpret_cast<uint32_t*>(op + x) = pack_bf16(v[x] * inv, v[x + 1] * inv);
            if (a.lse && lane == 0) {
              const int64_t at = a.cu ? h * a.rows + t : (bb * a.Hq + h) * a.T + ii;
              a.lse[at] = (st.x + log2f(st.z)) * 0.69314718055994530942f;
            }
          } else {
            const int64_t at = (static_cast<int64_t>(it.part) * a.rows + t) * a.Hq + h;
            if (st.z != 0.f) {  // NaN goes through
              float* op = a.part_o + at * D + lane * (D / 32);
#pragma unroll
              for (int x = 0; x < D / 32; x += 2)
                *reinterpret_cast<float2*>(op + x) = make_float2(v[x], v[x + 1]);
            }
            if (lane == 0) a.part_ml[at] = st;
          }
        }
        // the next row tile's copies (async proxy) may overwrite ob (generic proxy)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (tok[e] < 0) continue;
          const int64_t t = tok[e];
          if (sole) {
            const int64_t bb = a.cu ? 0 : t / a.T, ii = a.cu ? t : t - bb * a.T;
            const float inv = lb[e] == 0.f ? 0.f : 1.f / lb[e];
            __nv_bfloat16* op = a.o + bb * a.o_b + ii * a.o_s + head[e] * a.o_h + (lane & 3) * 2;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<uint32_t*>(op + n * 8) =
                  pack_bf16(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
            if (a.lse && (lane & 3) == 0) {
              const int64_t at = a.cu ? head[e] * a.rows + t : (bb * a.Hq + head[e]) * a.T + ii;
              a.lse[at] = (m[e] + log2f(lf[e])) * 0.69314718055994530942f;
            }
          } else {
            const int64_t at = (static_cast<int64_t>(it.part) * a.rows + t) * a.Hq + head[e];
            if (lf[e] != 0.f) {
              float* op = a.part_o + at * D + (lane & 3) * 2;
#pragma unroll
              for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(op + n * 8) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
            }
            if ((lane & 3) == 0) a.part_ml[at] = make_float4(m[e], lb[e], lf[e], 0.f);
          }
        }
      }
    }
  }
}

// Joins the parts of a row: one warp per (row, head), parts in order.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t x = blockIdx.x * int64_t(8) + (threadIdx.x >> 5);
  const int64_t t = x / a.Hq;
  const int h = static_cast<int>(x - t * a.Hq);
  if (t >= a.rows) return;
  if (a.cu && (t >= a.cu[a.B] || t < a.cu[0])) return;  // rows of no sequence stay as they are
  const int parts = a.splits_p + a.splits_o;
  const int64_t step = a.rows * a.Hq;
  const int64_t at = t * a.Hq + h;
  float M = -INFINITY;
  for (int p = lane; p < parts; p += 32) {
    const float4 v = a.part_ml[p * step + at];
    if (v.z != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float lb = 0.f, lf = 0.f;
  for (int p = 0; p < parts; ++p) {
    const float4 v = a.part_ml[p * step + at];
    if (v.z == 0.f) continue;
    const float w = ex2_approx(v.x - M);
    lb += w * v.y;
    lf += w * v.z;
    const float* op = a.part_o + (p * step + at) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * op[e];
  }
  const float inv = lb == 0.f ? 0.f : 1.f / lb;  // no key in sight: zeros
  const int64_t bb = a.cu ? 0 : t / a.T, ii = a.cu ? t : t - bb * a.T;
  __nv_bfloat16* op = a.o + bb * a.o_b + ii * a.o_s + h * a.o_h + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(op + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) {
    const int64_t li = a.cu ? h * a.rows + t : (bb * a.Hq + h) * a.T + ii;
    a.lse[li] = (M + log2f(lf)) * 0.69314718055994530942f;
  }
}

template <int D, int MT>
cudaError_t launch_one(const PagedArgs& a, const CUtensorMap& km, const CUtensorMap& vm,
                       cudaStream_t stream) {
  using L = PLayout<D, MT>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&attn_paged_kernel<D, MT>),
                                   L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(a.Hkv) *
                    ((a.splits_x ? 0 : static_cast<int64_t>(a.splits_p) * a.tiles_p) +
                     static_cast<int64_t>(a.splits_o) * a.tiles_o * a.B);
  if (n > 0x7fffffff) return cudaErrorInvalidValue;
  launch_begin(13, stream);
  attn_paged_kernel<D, MT><<<static_cast<unsigned>(n), kThreads, L::kBytes, stream>>>(km, vm, a);
  e = cudaGetLastError();
  launch_end(13, stream);
  return e;
}

}  // namespace

namespace {
// Rows beyond which the prefix goes to the tensor-core kernel with 128-row tiles.
bool prefix_on_tc(const PagedArgs& a) { return a.prefix >= 128 && a.rows * a.G > 16; }
bool small_tiles(const PagedArgs& a, int64_t max_q) {
  return max_q * a.G <= 16 && (a.prefix == 0 || a.splits_x || a.rows * a.G <= 16);
}
}  // namespace

void plan_paged(PagedArgs* a, int64_t max_q, int64_t max_len) {
  const int64_t rows_o = max_q * a->G, rows_p = a->rows * a->G;
  constexpr int kSms = 152;
  a->splits_x = 0;
  if (prefix_on_tc(*a)) {
    // One CTA per SM: waves of items, each as long as its share of key tiles and about four
    // tiles' time of start and end. The fewest splits of the shortest time.
    const bool pair = rows_p > 128;
    a->tiles_p = static_cast<int>((rows_p + (pair ? 255 : 127)) / (pair ? 256 : 128));
    const int64_t items = static_cast<int64_t>(a->tiles_p) * a->Hkv;
    const int64_t nt = (a->prefix + 127) / 128;
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s <= nt && s <= 160; ++s) {
      const int64_t waves = (items * s + kSms - 1) / kSms;
      const int64_t cost = waves * ((nt + s - 1) / s + 4);
      if (cost < best) {
        best = cost;
        a->splits_x = static_cast<int>(s);
      }
      if (waves > 16) break;
    }
    a->splits_p = a->splits_x * (pair ? 1 : 2);
  }
  const int MT = small_tiles(*a, max_q) ? 16 : 64;
  a->tiles_o = static_cast<int>((rows_o + MT - 1) / MT);
  const int64_t slots = 4 * kSms;  // two blocks on each SM, twice over
  auto splits = [&](int64_t items, int64_t keys) -> int {
    const int64_t nt = (keys + 255) / 256;
    int64_t s = (slots + items - 1) / items;
    if (s > nt) s = nt;
    return static_cast<int>(s < 1 ? 1 : s);
  };
  if (!a->splits_x) {
    a->tiles_p = static_cast<int>((rows_p + MT - 1) / MT);
    a->splits_p = a->prefix ? splits(static_cast<int64_t>(a->tiles_p) * a->Hkv, a->prefix) : 0;
  }
  a->splits_o = splits(static_cast<int64_t>(a->tiles_o) * a->Hkv * a->B, max_len);
}

cudaError_t launch_attn_paged(const PagedArgs& a, const CUtensorMap& k_map,
                              const CUtensorMap& v_map, int64_t max_q, cudaStream_t stream) {
  const bool small = small_tiles(a, max_q);
  if (a.D == 128)
    return small ? launch_one<128, 16>(a, k_map, v_map, stream)
                 : launch_one<128, 64>(a, k_map, v_map, stream);
  return small ? launch_one<64, 16>(a, k_map, v_map, stream)
               : launch_one<64, 64>(a, k_map, v_map, stream);
}

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
  const int64_t blocks = (a.rows * a.Hq + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  launch_begin(14, stream);
  if (a.D == 128) paged_merge_kernel<128><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  else paged_merge_kernel<64><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  launch_end(14, stream);
  return e;
}

}  // namespace upipe
