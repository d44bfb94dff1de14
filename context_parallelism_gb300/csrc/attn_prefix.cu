// The shared prefix of a paged-attention call on the 5th-generation tensor cores: all rows of the
// batch (the G q-heads of every new token) against the prefix's keys, per kv-head.
//
// Method, parts and statistics as in attn_paged.cu. A CTA holds up to two 128-row tiles or key
// streams, each with its softmax warpgroup (thread = row = TMEM lane), so that one's softmax
// overlaps the other's products:
//   kPair:  two row tiles walk the same key tiles (more than 128 rows): per key tile 64 KiB of
//           K and V feed 4 x 256 x 128 x D FLOP, and the tensor pipe sets the speed;
//   else:   one row tile (at most 128 rows), the even and the odd key tiles as two streams with
//           their own running statistics, joined at the end. HBM sets the speed.
//   S_w = Q_w K_j^T          tcgen05 (M 128, N 128, K D) -> TMEM S[w]
//   P_w = exp2(S_w c - m_w)  bf16, over S[w]'s first 64 columns
//   O_w += P_w V_j           tcgen05 with A from TMEM
// One warp issues every product. Where P lies over S, PV_w(j) goes before S_w's next tile, so the
// commit that publishes that S also says that O_w is settled and may be rescaled. With two row tiles
// of D 64 tensor memory has room for P beside S: then S_w's next tile is computed while this one's
// weights are (65536 keys, 128 sequences x 2 tokens, 64 q-heads: 384 -> 348 us). D 128 has that
// room only with 64-key tiles, whose smaller products cost more than they hide (877 -> 1200 us for
// 96 x 5 tokens on 131000 keys), as does Q in tensor memory there (1390 us), and as do two products
// of 64 keys a tile, the first one's columns filled while P lies over the second's (1103 us). What bounds two row
// tiles of D 128: the chain of one of them, its softmax (about 1500 cycles), its two products (1200)
// and the waits between them (700); the other one's runs in its gaps. Two threads a row (875 -> 929
// us) and scores read 32 columns at a time (949 us: each read waits behind the products' traffic to
// tensor memory) made the chain no shorter.
//
// Threads: warps 0-3 and 4-7 softmax (and the load of Q), warp 8 products, warp 9 (and 10) TMA: one
// lane per box of page rows, its page looked up while the stage is still in use.
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"

namespace upipe {
namespace {

// Two row tiles: ten warps; two key streams: eleven, K and V with a TMA warp each (one warp that
// issues both held 16-token pages to 402 us for 2.1 GB, against 335; where the tensor pipe sets
// the speed the eleventh warp costs 5 %).
constexpr int threads(bool pair) { return pair ? 320 : 352; }
// A row's weights are exp2(s - m) with m some 24 above the largest score of its first tile: below
// 2^-24 then, where a float and a bf16 are as exact as near 1. (Only products with values below some
// 2^-110 leave a float's normal range: rows of nothing but values of 1e-34 came out as exact as others,
// of 1e-36 5 % off.) m need not follow the maximum, so a tile's weights wait for no maximum of their
// own; a tile whose weights sum to more than 1 (its maximum is 17 or more above what m was made from)
// is done again with a new m, and O and the sums are scaled. Taking every tile's maximum first, and rescaling from 8 above m on, held 96 x 5 tokens
// on 131000 keys, where a few keys stand out, to 890 us against 850.
constexpr float kHeadroom = 24.0f;
constexpr float kLargeSum = 1.0f;
constexpr float kLowest = -3.0e38f;  // m of a row that has only -inf so far: any score is done again

template <int D, bool kPair>
struct XLayout {
  // P in columns of its own, where tensor memory has room for them (two row tiles of D 64)
  static constexpr bool kOwnP = kPair && D == 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQTiles = kPair ? 2 : 1;
  static constexpr int kStages = D == 128 ? (kPair ? 2 : 3) : (kPair ? 5 : 6);
  static constexpr int kQ = 0;
  static constexpr int kK = kQTiles * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kBar = kV + kStages * kTile;
  static constexpr int kNumBars = 1 + 4 * kStages + 2 + 2 + 2 + 2 + 1;
  static constexpr int kSlot = kBar + kNumBars * 8;
  static constexpr int kAbort = kSlot + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  // TMEM columns: S[2], P[2] (two bf16 a column) if it is not over S, O[2]
  static constexpr int tP = kOwnP ? 256 : 0, tPStep = kOwnP ? 64 : 128;
  static constexpr int tO = kOwnP ? 384 : 256;
  static_assert(tO + 2 * D <= 512, "tensor memory has 512 columns");
};

template <int D, bool kPair, bool kLse>
__global__ void __launch_bounds__(threads(kPair), 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using L = XLayout<D, kPair>;
  constexpr int NS = L::kStages;
  constexpr int kTile = L::kTile;
  constexpr bool kOwnP = L::kOwnP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* k_full = q_full + 1;
  uint64_t* v_full = k_full + NS;
  uint64_t* k_empty = v_full + NS;
  uint64_t* v_empty = k_empty + NS;
  uint64_t* s_full = v_empty + NS;  // [2]
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* o_done = p_full + 2;    // [2] with P in its own columns after every PV_w, else the last
  uint64_t* s_free = o_done + 2;    // [2] with P in its own columns: S_w is in registers
  uint64_t* drain = s_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();

  // kv-heads of one key range are neighbours (they read neighbouring bytes of the same pages),
  // then row blocks (the same bytes, from L2), then key ranges.
  int64_t x = blockIdx.x;
  const int kvh = static_cast<int>(x % a.Hkv);
  x /= a.Hkv;
  const int64_t row0 = (x % a.tiles_p) * (kPair ? 256 : 128);
  const int split = static_cast<int>(x / a.tiles_p);
  const int64_t n_rows = a.rows * a.G;
  const bool two = kPair ? row0 + 128 < n_rows : true;  // the second tile / stream has work
  const int64_t nt = (a.prefix + 127) / 128;
  const int64_t t_lo = nt * split / a.splits_x, t_hi = nt * (split + 1) / a.splits_x;
  const int n_kt = static_cast<int>(t_hi - t_lo);
  const int64_t k0 = t_lo * 128;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(v_full + i, 1);
      mbar_init(k_empty + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
      mbar_init(s_free + i, 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
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
          atomicOr(a.err, kErrWaitTimeout | 0x20000u);
          return false;
        }
      }
    }
  };

  if (warp >= 9) {
    // ---------------- TMA: K and V (warp 9), or K (warp 9) and V (warp 10) ----------------
    const int bx = a.box_rows;
    const int boxes = 128 / bx * (D / 64);  // at most 16
    const int r = lane / (D / 64) * bx, half = lane % (D / 64);
    const bool mine = lane < boxes;
    const uint32_t off = smem_u32(smem) + half * kBoxBytes + r * 128;
    const bool do_k = kPair || warp == 9, do_v = kPair || warp == 10;
    int issued_k = 0, issued_v = 0;
    bool ok = true;
    // one lane polls for the warp
    auto wait_one = [&](uint64_t* br, uint32_t parity) -> bool {
      int done = 1;
      if (lane == 0) done = wait(br, parity);
      return __shfl_sync(0xffffffffu, done, 0) != 0;
    };
    for (int j = 0; ok && j < n_kt; ++j) {
      const int s = j % NS;
      const uint32_t ph = (j / NS - 1) & 1;
      // A box past the prefix, or of a page that does not exist, lies outside the tensor map and
      // reads as zeros; nothing outside the caches is touched.
      int page = -1, slot = 0;
      const int64_t key = k0 + static_cast<int64_t>(j) * 128 + r;
      if (mine && key < a.prefix) {
        const int64_t pg = key / a.page_size;
        page = a.ptable[pg];
        slot = static_cast<int>(key - pg * a.page_size);
        if (page < 0 || page >= a.n_pages) {
          page = -1;
          atomicOr(a.err, kErrBadPage);
        }
      }
      if (do_k) {
        if (j >= NS) ok = wait_one(k_empty + s, ph);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(k_full + s, kTile);
        __syncwarp();
        if (mine) tma_load_4d(off + L::kK + s * kTile, &tm_k, half * 64, slot, kvh, page, k_full + s);
        issued_k = j + 1;
      }
      if (do_v) {
        if (j >= NS) ok = wait_one(v_empty + s, ph);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(v_full + s, kTile);
        __syncwarp();
        if (mine) tma_load_4d(off + L::kV + s * kTile, &tm_v, half * 64, slot, kvh, page, v_full + s);
        issued_v = j + 1;
      }
    }
    if (!ok) {  // copies in flight land before the CTA's shared memory goes
      for (int j = issued_k > NS ? issued_k - NS : 0; j < issued_k; ++j)
        mbar_wait(k_full + j % NS, (j / NS) & 1, 100000000ull);
      for (int j = issued_v > NS ? issued_v - NS : 0; j < issued_v; ++j)
        mbar_wait(v_full + j % NS, (j / NS) & 1, 100000000ull);
    }
  } else if (warp == 8) {
    // ---------------- products ----------------
    // The warp stays converged, one lane issues: operands in uniform registers.
    {
      auto wait_all = [&](uint64_t* br, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(br, parity));
      };
      const uint32_t id_s = idesc_bf16(128, 128, false, false);
      const uint32_t id_o = idesc_bf16(128, D, false, true);
      const uint64_t base_k = kdesc0(smem_u32(smem));
      const uint64_t base_mn = mndesc0(smem_u32(smem));
      constexpr uint32_t kTileU = kTile >> 4;
      bool ok = wait_all(q_full, 0);
      auto issue_s = [&](int w, int j) -> bool {
        const int s = j % NS;
        if ((!kPair || w == 0) && !wait_all(k_full + s, (j / NS) & 1)) return false;
        if (kOwnP && j > 0 && !wait_all(s_free + w, (j - 1) & 1)) return false;
        tc_fence_after();
        const uint64_t bk = base_k;
        const uint32_t uq = (L::kQ >> 4) + (kPair ? w * kTileU : 0u);
        const uint32_t uk = (L::kK >> 4) + s * kTileU;
#pragma unroll
        for (int k16 = 0; k16 < D / 16; ++k16)
          umma_f16_ss_warp(tmem + 128 * w, bk + (uq + kstep(k16)), bk + (uk + kstep(k16)), id_s,
                           k16 > 0 ? 1u : 0u);
        umma_commit_warp(s_full + w);
        if (!kPair || w == 1 || !two) umma_commit_warp(k_empty + s);
        return true;
      };
      // n: how many tiles tile/stream w has taken before this one
      auto issue_pv = [&](int w, int j, int n, bool last) -> bool {
        const int s = j % NS;
        if (!wait_all(p_full + w, n & 1)) return false;
        if ((!kPair || w == 0) && !wait_all(v_full + s, (j / NS) & 1)) return false;
        tc_fence_after();
        const uint64_t bmn = base_mn;
        const uint32_t uv = (L::kV >> 4) + s * kTileU;
#pragma unroll
        for (int k16 = 0; k16 < 8; ++k16)
          umma_f16_ts_warp(tmem + L::tO + D * w, tmem + L::tP + L::tPStep * w + k16 * 8,
                           bmn + (uv + mnstep(k16)), id_o, (k16 > 0 || n > 0) ? 1u : 0u);
        if (kOwnP || last) umma_commit_warp(o_done + w);
        if (!kPair || w == 1 || !two) umma_commit_warp(v_empty + s);
        return true;
      };
      if (kOwnP) {
        // S_w(j + 1) as soon as S_w(j) is in registers, while its weights are computed; in the
        // order in which the two groups, half a tile apart, are ready
        if (ok && n_kt > 0) ok = issue_s(0, 0) && (!two || issue_s(1, 0));
        for (int j = 0; ok && j < n_kt; ++j) {
          const bool more = j + 1 < n_kt;
          if (more) ok = issue_s(0, j + 1);
          if (ok && two && j > 0) ok = issue_pv(1, j - 1, j - 1, false);
          if (ok && two && more) ok = issue_s(1, j + 1);
          if (ok) ok = issue_pv(0, j, j, !more);
        }
        if (ok && two && n_kt > 0) ok = issue_pv(1, n_kt - 1, n_kt - 1, true);
      } else if (kPair) {
        if (ok && n_kt > 0) ok = issue_s(0, 0) && (!two || issue_s(1, 0));
        for (int j = 0; ok && j < n_kt; ++j) {
          const bool more = j + 1 < n_kt;
          ok = issue_pv(0, j, j, !more);
          if (ok && more) ok = issue_s(0, j + 1);
          if (ok && two) ok = issue_pv(1, j, j, !more);
          if (ok && two && more) ok = issue_s(1, j + 1);
        }
      } else {
        if (ok && n_kt > 0) ok = issue_s(0, 0);
        if (ok && n_kt > 1) ok = issue_s(1, 1);
        for (int j = 0; ok && j < n_kt; ++j) {
          ok = issue_pv(j & 1, j, j >> 1, j + 2 >= n_kt);
          if (ok && j + 2 < n_kt) ok = issue_s(j & 1, j + 2);
        }
      }
      if (!ok) {
        umma_commit_warp(drain);
        mbar_wait(drain, 0, 100000000ull);
      }
    }
  } else {
    // ---------------- Q, softmax ----------------
    {
      // a thread loads one 16-byte chunk of every kStep-th row, eight rows in flight
      constexpr int kChunks = D / 8, kStep = 256 / kChunks, kRows = L::kQTiles * 128;
      const int c = threadIdx.x % kChunks;
      const uint32_t G = a.G, T = static_cast<uint32_t>(a.T);
#pragma unroll 1
      for (int r0 = threadIdx.x / kChunks; r0 < kRows; r0 += 8 * kStep) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t row = row0 + r0 + u * kStep;
          v[u] = make_uint4(0, 0, 0, 0);
          if (r0 + u * kStep < kRows && row < n_rows) {
            const uint32_t t = static_cast<uint32_t>(row) / G;
            const int h = kvh * a.G + static_cast<int>(static_cast<uint32_t>(row) - t * G);
            const uint32_t bb = a.cu ? 0 : T == 1 ? t : t / T, ii = a.cu ? t : t - bb * T;
            v[u] = *reinterpret_cast<const uint4*>(a.q + bb * a.q_b + ii * a.q_s + h * a.q_h + c * 8);
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = r0 + u * kStep;
          if (r < kRows)
            st_shared_v4(smem_u32(smem) + L::kQ + (r >> 7) * kTile + swz_offset(r & 127, c * 8),
                         v[u].x, v[u].y, v[u].z, v[u].w);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int w = warp >> 2;
    const int t128 = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * w, tP = tmem + L::tP + L::tPStep * w, tO = tmem + L::tO + D * w;
    const int64_t row = row0 + (kPair ? 128 * w : 0) + t128;
    // a warp without rows only keeps the barriers going: its TMEM lanes reach no output
    const bool work = row - (threadIdx.x & 31) < n_rows;
    float m_used = -INFINITY, lb = 0.f, lf = 0.f;
    // the scores are in registers: S_w may be overwritten with the next tile's
    auto s_read = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free + w);
    };
    bool good = true;
    int n = 0;
    const int j0 = kPair ? 0 : w, dj = kPair ? 1 : 2;
    const int n_mine = kPair && w == 1 && !two ? 0 : n_kt;
    for (int j = j0; j < n_mine; j += dj, ++n) {
      good = __all_sync(0xffffffffu, wait(s_full + w, n & 1));
      if (!good) break;
      tc_fence_after();
      const int64_t key0 = k0 + static_cast<int64_t>(j) * 128;
      const int valid = key0 + 128 > a.prefix ? static_cast<int>(a.prefix - key0) : 128;
      if (valid < 128 && (!kPair || w == 0)) {
        // values in slots past the prefix may be anything, and 0 * NaN is not 0: cleared before
        // the product reads them (this group's arrival on p_full publishes the stores)
        const int s = j % NS;
        good = __all_sync(0xffffffffu, wait(v_full + s, (j / NS) & 1));
        if (!good) break;
        for (int i = t128; i < (128 - valid) * (D / 8); i += 128)
          st_shared_v4(smem_u32(smem) + L::kV + s * kTile +
                           swz_offset(valid + i / (D / 8), i % (D / 8) * 8),
                       0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      if (work) {
        float alpha = 1.f;
        bool upd = false;
        uint32_t ra[64], rb[64];
        float sum;
        uint64_t f0, f1;  // pairs of sums of the fp32 weights, for lse alone
        bool fresh = n == 0;  // m is to be made
        while (true) {
          tmem_ld64_nowait(tS + lane_off + 64, rb);
          tmem_ld64_nowait(tS + lane_off, ra);
          tmem_wait_ld_dep64(ra);
          tmem_reg_dep64(rb);
          if (valid < 128) {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              if (i >= valid) ra[i] = __float_as_uint(-INFINITY);
              if (64 + i >= valid) rb[i] = __float_as_uint(-INFINITY);
            }
          }
          if (fresh) {
            float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 64; ++i)
              mq[i & 3] = fmax3(mq[i & 3], __uint_as_float(ra[i]), __uint_as_float(rb[i]));
            const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
            const float to = fmaxf(mx * a.scale_log2 + kHeadroom, kLowest);
            if (to > m_used) {
              alpha = ex2_approx(m_used - to);
              m_used = to;
              upd = true;
            }
          }
          const uint64_t sl2 = f2_pack(a.scale_log2, a.scale_log2);
          const uint64_t nm2 = f2_pack(-m_used, -m_used);
          float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
          f0 = f1 = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x0, x1;
            f2_unpack(ffma2(f2_pack_u(ra[2 * i], ra[2 * i + 1]), sl2, nm2), x0, x1);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            if (kLse) f0 = fadd2(f0, f2_pack(e0, e1));
            ra[i] = pack_bf16(e0, e1);
            add_bf16x2(sa[2 * (i & 1)], sa[2 * (i & 1) + 1], ra[i]);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x0, x1;
            f2_unpack(ffma2(f2_pack_u(rb[2 * i], rb[2 * i + 1]), sl2, nm2), x0, x1);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            if (kLse) f1 = fadd2(f1, f2_pack(e0, e1));
            rb[i] = pack_bf16(e0, e1);
            add_bf16x2(sb[2 * (i & 1)], sb[2 * (i & 1) + 1], rb[i]);
          }
          sum = ((sa[0] + sa[1]) + (sb[0] + sb[1])) + ((sa[2] + sa[3]) + (sb[2] + sb[3]));
          if (fresh || !__any_sync(0xffffffffu, sum > kLargeSum)) break;
          fresh = true;
        }
        if constexpr (kOwnP) s_read();
        lb = lb * alpha + sum;
        if (kLse) {
          float g0, g1;
          f2_unpack(fadd2(f0, f1), g0, g1);
          lf = lf * alpha + (g0 + g1);
        }
        // P's own columns and O are free once PV_w of the tile before has run
        if (kOwnP && n > 0) {
          good = __all_sync(0xffffffffu, wait(o_done + w, (n - 1) & 1));
          if (!good) break;
          tc_fence_after();
        }
        {
          uint32_t pa[32], pb[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            pa[i] = ra[i];
            pb[i] = rb[i];
          }
          tmem_st32(tP + lane_off, pa);
          tmem_st32(tP + lane_off + 32, pb);
        }
        if (n > 0 && __any_sync(0xffffffffu, upd)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tmem_ld32_sync(tO + lane_off + c * 32, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st32(tO + lane_off + c * 32, r);
          }
        }
        tmem_wait_st();
      } else {
        if constexpr (kOwnP) {
          s_read();
          // as the others: no arrival on p_full for this tile before the one before it is complete
          if (n > 0) good = __all_sync(0xffffffffu, wait(o_done + w, (n - 1) & 1));
          if (!good) break;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + w);
    }
    if (good && n > 0) {
      good = __all_sync(0xffffffffu, wait(o_done + w, kOwnP ? (n - 1) & 1 : 0));
      if (good) tc_fence_after();
    }
    if (good && work) {
      const int part = kPair ? split : 2 * split + w;
      if (!kLse) lf = lb;
      const int64_t t = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.G);
      const int h = kvh * a.G + static_cast<int>(row - t * a.G);
      const int64_t at = (static_cast<int64_t>(part) * a.rows + t) * a.Hq + h;
      const bool row_ok = row < n_rows;
      if (n > 0) {
        float* op = a.part_o + at * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          tmem_ld32_sync(tO + lane_off + c * 32, r);
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) st_global_v8(op + c * 32 + i, &r[i]);
          }
        }
      }
      if (row_ok) a.part_ml[at] = make_float4(m_used, lb, lf, 0.f);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kPair, bool kLse>
cudaError_t launch_one(const PagedArgs& a, const CUtensorMap& km, const CUtensorMap& vm,
                       cudaStream_t stream) {
  using L = XLayout<D, kPair>;
  cudaError_t e = ensure_smem_attr(
      reinterpret_cast<const void*>(&attn_prefix_kernel<D, kPair, kLse>), L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t n = static_cast<int64_t>(a.Hkv) * a.tiles_p * a.splits_x;
  if (n > 0x7fffffff) return cudaErrorInvalidValue;
  launch_begin(15, stream);
  attn_prefix_kernel<D, kPair, kLse><<<static_cast<unsigned>(n), threads(kPair), L::kBytes, stream>>>(km, vm, a);
  e = cudaGetLastError();
  launch_end(15, stream);
  return e;
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, const CUtensorMap& km, const CUtensorMap& vm,
                     cudaStream_t stream) {
  if (a.rows * a.G > 128)
    return a.lse ? launch_one<D, true, true>(a, km, vm, stream)
                 : launch_one<D, true, false>(a, km, vm, stream);
  return a.lse ? launch_one<D, false, true>(a, km, vm, stream)
               : launch_one<D, false, false>(a, km, vm, stream);
}

}  // namespace

cudaError_t launch_attn_prefix(const PagedArgs& a, const CUtensorMap& k_map,
                               const CUtensorMap& v_map, cudaStream_t stream) {
  return a.D == 128 ? launch_d<128>(a, k_map, v_map, stream) : launch_d<64>(a, k_map, v_map, stream);
}

}  // namespace upipe
