// Attention of a batch's new tokens over a paged key/value cache: the prefix that the whole batch
// shares (where attn_prefix.cu does not take it) and each sequence's own pages.
//
// Row (sequence b, new token i of n, q-head h) sees the prefix's keys 0..P-1 and its own keys
// 0..len_b - n + i. Per kv-head, a segment is a tile of rows (the G q-heads of consecutive
// tokens; of all sequences for the prefix, of one for its own pages) with all its keys:
//   s = scale <q, k>,  m = max s,  p = exp2(s - m) (log2 units),  O~ = sum p v,  l = sum p,
// one pass with the running maximum and sum. A segment may be cut along its keys; each piece's
// (m, l, O~) is one part of its rows, and the parts of a row are joined by
//   M = max m_p,  o = sum 2^(m_p - M) O~_p / sum 2^(m_p - M) l_p,  lse = ln 2 (M + log2 l).
// P is rounded to bf16 for the P V product. Two sums are kept: that of the rounded weights
// divides O~ (numerator and denominator agree), that of the fp32 weights gives lse.
//
// Bound: HBM (each key and value is read once per row tile; 4 bytes per key feature carry
// 4 x rows FLOP). The matrix instruction is mma.sync m16n8k16: a decode step has G to 16 rows a
// kv-head, which a 128-row tcgen05 tile would fill to an eighth at most.
//
// Shares. The key tiles of all segments, in order, are cut into equal shares, one per worker:
// lengths are read on the device, so ragged batches and captured graphs whose lengths move stay
// balanced. A worker's share is a run of pieces of neighbouring segments; the piece of segment g
// at worker c is kept in slot g + c (each step along the run moves g or c by one, so slots are
// distinct, and a segment's pieces are neighbours). Segments are numbered sequence, row tile,
// kv-head: neighbouring workers read neighbouring heads of the same pages.
//
// Two kernels, by the rows that a sequence has for a kv-head:
//   up to 16 (a decode step): a worker is a single warp with a ring of stages of its own;
//   17 and more: a worker is a block of one producer warp and four consumer warps of 16 rows.
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"

namespace upipe {
namespace {

constexpr int kSms = 152;

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
// Transpose of an 8 x 8 matrix of 16-bit elements, two per lane in row-major lane order.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What is to be known of a piece to compute it.
struct Piece {
  int64_t tok0;      // first row of q of the segment's group
  int64_t slot;
  int32_t row0;      // first row (token, head-of-group order) of the tile
  int32_t n_rows;    // rows of the group
  int32_t kvh, own;  // own: the keys are the sequence's own (causal limit)
  int32_t n_kt;      // tiles; -1: no more pieces
  int32_t keys;      // keys of the piece
  int32_t before;    // keys of the piece that token 0 sees, less one (own pieces; clamped)
  int32_t parts;     // pieces of the segment
  int32_t first;     // this one is its first
};

static_assert(sizeof(Piece) % 8 == 0, "pieces keep the alignment of their words");

// What starting and ending a piece costs, in tiles: each segment counts as so many tiles more, so
// that a worker with many short sequences has fewer keys. Tile t of a segment is at kOver + t.
constexpr uint32_t kOver = kSegmentCost;

// One group of segments (the prefix: b = -1, or a sequence): its rows and keys.
struct Group {
  int tok0, n_tok;   // rows of q
  int keys;          // that the table holds
  int len;           // own tokens as given: more than keys where the table is too narrow
  uint32_t segs;     // row tiles x kv-heads
  uint32_t cost;     // kOver + tiles per segment, at least one (a segment without keys still writes)
  __device__ __forceinline__ uint32_t tiles() const { return segs * cost; }  // host: below 2^32
};

template <int KS, int MT>
__device__ __forceinline__ Group load_group(const PagedArgs& a, int b, bool report) {
  Group g;
  const int rows = static_cast<int>(a.rows);
  if (b < 0) {
    g.tok0 = 0;
    g.n_tok = a.splits_x || !a.prefix ? 0 : a.cu ? min(rows, max(a.cu[a.B], 0)) : rows;
    g.len = g.keys = static_cast<int>(a.prefix);
  } else {
    const int len = a.seq_len[b];
    if (a.cu) {
      const int c0 = a.cu[b], c1 = a.cu[b + 1];
      g.tok0 = min(max(c0, 0), rows);
      g.n_tok = max(min(c1, rows) - g.tok0, 0);
    } else {
      g.tok0 = b * static_cast<int>(a.T);
      g.n_tok = static_cast<int>(a.T);
    }
    if (report && len > a.cap) atomicOr(a.err, kErrBadPage);
    g.len = max(len, 0);
    g.keys = min(g.len, a.cap);
  }
  g.segs = (static_cast<uint32_t>(g.n_tok * a.G) + (MT - 1)) / MT * a.Hkv;
  g.cost = kOver + max((static_cast<uint32_t>(g.keys) + (KS - 1)) / KS, 1u);
  return g;
}

// A place in a worker's share; every lane of the warp holds the same.
template <int KS, int MT>
struct Walk {
  Group g;
  uint32_t left, share;      // tiles that are still to come, and of a whole share
  uint32_t group_seg, seg, kt;  // segments before the group; segment of the group, tile of it
  int b, worker, kvh, row0;
  int k_lo, k_hi;            // the piece's keys

  // Cuts all tiles into the workers' shares (of at least `least` tiles) and finds this worker's
  // start. Sequences are taken 32 at a time, one per lane. A block has up to `most` workers, and
  // as many as are needed, so that few shares go to as many SMs; the workers of a block take
  // neighbouring shares.
  // first: what the first two rounds load (sequences lane and lane + 32), asked for at the
  // kernel's very start, before anything that a load cannot pass.
  struct First {
    Group g[2];
  };
  __device__ __forceinline__ static First begin(const PagedArgs& a, int lane, bool report) {
    First f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f.g[i].segs = f.g[i].cost = 0;
      if (lane + 32 * i < a.B) f.g[i] = load_group<KS, MT>(a, lane + 32 * i, report);
    }
    return f;
  }
  __device__ __forceinline__ void init(const PagedArgs& a, int lane, uint32_t in_block,
                                       uint32_t most, uint32_t least, const First& first) {
    left = group_seg = seg = kt = 0;
    kvh = row0 = worker = 0;
    b = -1;
    Group mine = first.g[0];  // the round's sequence of this lane
    g = load_group<KS, MT>(a, -1, false);
    uint32_t total = mine.tiles() + first.g[1].tiles();
    for (int b0 = lane + 64; b0 < a.B; b0 += 32)
      total += load_group<KS, MT>(a, b0, blockIdx.x == 0 && in_block == 0).tiles();
#pragma unroll
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    total += g.tiles();
    if (total == 0) return;
    uint32_t per_block = most;
    if (total < static_cast<uint64_t>(least) * gridDim.x * most)
      per_block = min(((total - 1) / least) / gridDim.x + 1, most);
    share = max((total - 1) / (gridDim.x * per_block) + 1, least);
    worker = static_cast<int>(blockIdx.x * per_block + in_block);
    if (in_block >= per_block || static_cast<uint64_t>(worker) * share >= total) return;
    uint32_t x = worker * share;
    left = min(share, total - x);
    if (x >= g.tiles()) {
      x -= g.tiles();
      group_seg = g.segs;
      for (int b0 = 0;; b0 += 32) {
        if (b0 == 32) {
          mine = first.g[1];
        } else if (b0 > 32) {
          mine.segs = mine.cost = 0;
          if (b0 + lane < a.B) mine = load_group<KS, MT>(a, b0 + lane, false);
        }
        uint32_t ws = mine.tiles(), ns = mine.segs;  // inclusive sums over the lanes
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, ws, s);
          const uint32_t v = __shfl_up_sync(0xffffffffu, ns, s);
          if (lane >= s) {
            ws += u;
            ns += v;
          }
        }
        const uint32_t past = __ballot_sync(0xffffffffu, ws > x);
        if (past) {
          const int l = __ffs(past) - 1;
          b = b0 + l;
          x -= __shfl_sync(0xffffffffu, ws - mine.tiles(), l);
          group_seg += __shfl_sync(0xffffffffu, ns - mine.segs, l);
          g.tok0 = __shfl_sync(0xffffffffu, mine.tok0, l);
          g.n_tok = __shfl_sync(0xffffffffu, mine.n_tok, l);
          g.len = __shfl_sync(0xffffffffu, mine.len, l);
          g.keys = min(g.len, a.cap);
          g.segs = __shfl_sync(0xffffffffu, mine.segs, l);
          g.cost = __shfl_sync(0xffffffffu, mine.cost, l);
          break;
        }
        x -= __shfl_sync(0xffffffffu, ws, 31);
        group_seg += __shfl_sync(0xffffffffu, ns, 31);
        if (b0 + 32 >= a.B) {  // not reached: the shares add up to the tiles
          left = 0;
          return;
        }
      }
    }
    seg = x / g.cost;
    kt = x - seg * g.cost;
    const uint32_t rt = seg / a.Hkv;
    kvh = static_cast<int>(seg - rt * a.Hkv);
    row0 = static_cast<int>(rt) * MT;
  }

  // The next piece; false at the end of the share.
  __device__ __forceinline__ bool next(const PagedArgs& a, Piece* p) {
    if (left == 0) return false;
    while (seg >= g.segs) {
      group_seg += g.segs;
      seg = 0;
      row0 = kvh = 0;
      if (++b >= a.B) return false;
      g = load_group<KS, MT>(a, b, false);
    }
    if (kt < kOver) {
      const uint32_t n = min(kOver - kt, left);
      kt += n;
      left -= n;
      if (left == 0) return false;
    }
    const uint32_t n = min(g.cost - kt, left), t0 = kt - kOver;
    k_lo = min(static_cast<int>(t0 * KS), g.keys);
    k_hi = static_cast<int>(min((t0 + n) * KS, static_cast<uint32_t>(g.keys)));
    p->tok0 = g.tok0;
    p->slot = static_cast<int64_t>(group_seg) + seg + worker;
    p->row0 = row0;
    p->n_rows = g.n_tok * a.G;
    p->kvh = kvh;
    p->own = b >= 0;
    p->keys = k_hi - k_lo;
    p->n_kt = (p->keys + KS - 1) / KS;
    p->before = g.len - g.n_tok - k_lo;
    p->first = t0 == 0;
    // workers from the segment's first tile to its last (known where the segment starts)
    const uint32_t rest = g.cost - kt - n;
    p->parts = t0 == 0 ? 1 + static_cast<int>(rest ? (rest + share - 1) / share : 0u) : 2;
    left -= n;
    kt += n;
    if (kt == g.cost) {
      kt = 0;
      ++seg;
      if (++kvh == a.Hkv) {
        kvh = 0;
        row0 += MT;
      }
    }
    return true;
  }
};

// Token and q-head of a tile's row, and its place in q, o and lse.
struct Row {
  int i, h;       // token of the group, q-head
  int64_t t;      // row of q
  int64_t b, s;   // batch row and place (packed rows: 0 and t)
};

__device__ __forceinline__ Row find_row(const PagedArgs& a, const Piece& p, int r) {
  Row w;
  const int row = p.row0 + r;
  // one token's rows, as in a plain decode step, need no division
  w.i = row < a.G ? 0 : static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(a.G));
  w.h = p.kvh * a.G + row - w.i * a.G;
  w.t = p.tok0 + w.i;
  if (a.cu) {
    w.b = 0;
    w.s = w.t;
  } else if (p.own) {  // the group is a batch row of T tokens
    w.s = w.i;
    w.b = a.T == 1 ? w.t : div_fl(p.tok0, a.T);
  } else {
    w.b = a.T == 1 ? w.t : div_fl(w.t, a.T);
    w.s = w.t - w.b * a.T;
  }
  return w;
}

// Where a row's results go: its own outputs if the piece is all that its row has, else its slot.
struct RowOut {
  __nv_bfloat16* o;
  float* lse;
  float* part;
  float4* ml;
};

// say: this lane tells the join where the row's pieces are.
__device__ __forceinline__ RowOut row_out(const PagedArgs& a, const Piece& p, int r, int MT, int D,
                                          bool say) {
  RowOut w = {nullptr, nullptr, nullptr, nullptr};
  const Row f = find_row(a, p, r);
  const bool sole = p.parts == 1 && a.prefix == 0;
  if (sole) {
    w.o = a.o + f.b * a.o_b + f.s * a.o_s + f.h * a.o_h;
    if (a.lse) w.lse = a.lse + (a.cu ? f.h * a.rows + f.t : (f.b * a.Hq + f.h) * a.T + f.s);
  } else if (p.slot < a.n_slots) {  // beyond only for cu_rows that decrease
    w.part = a.slot_o + (p.slot * MT + r) * D;
    w.ml = a.slot_ml + (p.slot * MT + r);
  }
  if (p.first && say)
    a.desc[(p.own ? a.rows * a.Hq : 0) + f.t * a.Hq + f.h] =
        make_int2(static_cast<int>(p.slot * MT + r), sole ? 0 : p.parts);
  return w;
}

__device__ __forceinline__ const __nv_bfloat16* q_row(const PagedArgs& a, const Piece& p, int r) {
  if (p.row0 + r >= p.n_rows) return nullptr;
  const Row f = find_row(a, p, r);
  return a.q + f.b * a.q_b + f.s * a.q_s + f.h * a.q_h;
}

// Keys of the piece that a row sees.
__device__ __forceinline__ int row_limit(const PagedArgs& a, const Piece& p, int r) {
  const int row = p.row0 + r;
  if (row >= p.n_rows) return 0;
  if (!p.own) return p.keys;
  const int i = row < a.G ? 0 : static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(a.G));
  return min(p.keys, p.before + i + 1);
}

template <typename T>
__device__ __forceinline__ T* shfl_ptr(T* p, int src) {
  return reinterpret_cast<T*>(
      __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), src));
}

// Values that some row of a tile must not see. A key beyond a row's causal limit has weight 0, and
// 0 * v is 0 only for a finite v: an infinity or NaN there (a later drafted token's) would reach
// rows that end before it. So where a limit lies inside the tile, its V is looked over from the
// first such key on, and if anything is not finite the tile's products are taken key by key, each
// row adding only what it sees.

// Whether rows [r0, KS) of a stage's V hold an infinity or NaN; the same in every lane.
template <int D, int KS>
__device__ __forceinline__ bool any_not_finite(uint32_t sv, int r0, int lane) {
  constexpr uint32_t kLo = 0x7f80u, kHi = 0x7f800000u;  // exponents of the two halves
  bool bad = false;
  for (int x = r0 * (D / 8) + lane; x < KS * (D / 8); x += 32) {
    const int r = x / (D / 8), ch = x % (D / 8);
    uint32_t w[4];
    ld_shared_v4(w, sv + (ch >> 3) * (KS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (w[i] & kLo) == kLo || (w[i] & kHi) == kHi;
  }
  return __any_sync(0xffffffffu, bad);
}

// Address of feature f (of an even pair) of row r in a stage's V.
template <int KS>
__device__ __forceinline__ uint32_t v_at(uint32_t sv, int r, int f) {
  return sv + (f >> 6) * (KS * 128) + r * 128 + ((((f >> 3) & 7) ^ (r & 7)) << 4) + (f & 7) * 2;
}

// ---- up to 16 rows: one warp a worker --------------------------------------------------------
//
// S^T = K Q^T and O^T += V^T P^T: keys and features fill the instruction's 16 rows, the few query
// rows its 8 columns (NR column tiles). The warp keeps its piece's rows in registers and issues
// the copies into its ring itself, each stage's next one as soon as it has read it, running on
// into the pieces that follow: no producer, no barrier but a stage's own, nothing to meet at.
constexpr int kWarps = 8;

template <int D, int NR>
struct DLayout {
  static constexpr int kKeys = 2048 / D;            // 8 KiB of K and V a stage
  static constexpr int kStage = 2 * kKeys * D * 2;
  static constexpr int kStages = 3;
  static constexpr int kPieces = 4;                 // published ahead: one a stage and one more
  static constexpr int kBar = kWarps * kStages * kStage;
  static constexpr int kPiece = kBar + kWarps * kStages * 8;
  static constexpr int kBytes = kPiece + kWarps * kPieces * static_cast<int>(sizeof(Piece)) + 1024;
};

// kSeveral: a sequence may have several new tokens, so a row may end before the others. With one token
// each no limit lies inside a tile, and the test for it is left out: it cost 1.5 % of 131072 keys. Where
// it is needed, the look at a sequence's last tiles costs 1.3 of 38.6 us (40 x 2 tokens, D 64); the
// weights computed on both sides of the branch, so that none stands before the products, gave the same.
template <int D, int NR, bool kSeveral>
__global__ void __launch_bounds__(kWarps * 32, 1)
    paged_decode_kernel(const __grid_constant__ PagedArgs a) {
  using L = DLayout<D, NR>;
  constexpr int MT = 8 * NR, KS = L::kKeys, NS = L::kStages;
  constexpr int kHalf = KS * 128;      // bytes of a stage's 64 features of K or V
  constexpr int kVoff = KS * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar) + warp * NS;
  Piece* pieces = reinterpret_cast<Piece*>(smem + L::kPiece) + warp * L::kPieces;
  const uint32_t ring = smem_u32(smem) + warp * NS * L::kStage;

  const auto first = Walk<KS, MT>::begin(a, lane, blockIdx.x == 0 && warp == 0);
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(full + i, 32);  // every lane's copies
  }
  {
    // the tables, on their way to L2 while the lengths are read
    const uint32_t line = blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t per = static_cast<uint32_t>(min((a.max_pages + 31) / 32, int64_t(1) << 20));
    const uint32_t b = line / per;
    if (b < static_cast<uint32_t>(a.B))
      prefetch_l2(a.table + b * a.table_stride + (line - b * per) * 32);
  }
  __syncwarp();

  // ---- the copies: a place in the share that runs ahead of the computation ----
  Walk<KS, MT> wk;
  wk.init(a, lane, warp, kWarps, static_cast<uint32_t>(a.least), first);
  // Copies are 16 bytes a lane (cp.async): a row of a page is D / 8 lanes, a warp instruction
  // kRows rows. Pages are looked up for 32 runs of 16 keys at a time, one a lane, so that a tile's
  // copies wait for no load. (TMA boxes of 16 page rows, the smallest page, moved a quarter less:
  // 2.1 GB of 16-token pages in 435 against 389 us.)
  constexpr int kChunks = D / 8, kRows = 32 / kChunks;
  const int c_row = lane / kChunks, c_col = lane % kChunks;
  const uint32_t dst0 = (c_col >> 3) * kHalf + c_row * 128 + (((c_col & 7) ^ c_row) << 4);
  const int64_t row_step = 2 * kRows * a.slot_stride;  // bytes
  const int64_t v_minus_k = reinterpret_cast<const char*>(a.vc) - reinterpret_cast<const char*>(a.kc);
  const char* k0_ptr = nullptr;  // this lane's part of a row of the piece's head
  uint32_t n_cp = 0, n_pc = 0;  // tiles copied and pieces published so far
  int left = 0;                 // tiles of the piece that are still to be copied
  int key0 = 0;
  int win = 0;                  // first key of the 32 runs looked up
  int64_t win_at = -1;          // this lane's: offset of the run's first row in the caches
  const int32_t* pages = nullptr;
  bool more = true;
  auto look_up = [&]() {
    static_assert(kMaxOwnKeys <= 0x7fffffff - 31 * 16, "a key behind the last one has a number");
    win = key0;
    const int key = key0 + lane * 16;
    win_at = -1;  // past the keys, or a page that does not exist: zeros
    if (key < wk.k_hi) {
      const uint32_t pg = static_cast<uint32_t>(key) / static_cast<uint32_t>(a.page_size);
      const int page = pages[pg];
      if (page >= 0 && page < a.n_pages)
        win_at = page * a.page_stride + (key - static_cast<int>(pg) * a.page_size) * a.slot_stride;
      else
        atomicOr(a.err, kErrBadPage);
    }
  };
  // Publishes the next piece (one without keys too).
  auto publish = [&]() {
    Piece p;
    more = wk.next(a, &p);
    if (!more) p.n_kt = -1;
    if (lane == 0) pieces[n_pc % L::kPieces] = p;
    __syncwarp();
    ++n_pc;
    left = more ? p.n_kt : 0;
    if (left == 0) return;
    key0 = wk.k_lo;
    k0_ptr = reinterpret_cast<const char*>(a.kc + p.kvh * a.head_stride + c_row * a.slot_stride +
                                           c_col * 8);
    pages = p.own ? a.table + wk.b * a.table_stride : a.ptable;
    look_up();
    // the piece's rows of q, on their way to L2 before they are needed: a load that has to wait
    // behind all the keys and values in flight takes microseconds
    constexpr int kLines = D / 64;
    if (lane < MT * kLines) {
      const __nv_bfloat16* qp = q_row(a, p, lane / kLines);
      if (qp) prefetch_l2(qp + lane % kLines * 64);
    }
  };
  // Copies the next tile into the stage that the tile kStages before it has left, publishing pieces
  // on the way as long as there is room for them; false if there is nothing to copy now. Rows past
  // the keys become zeros (whatever their slots hold: 0 * inf is not 0), and nothing outside the
  // caches is touched.
  auto copy_next = [&](uint32_t n_done) -> bool {
    while (left == 0) {
      if (!more || n_pc - n_done >= static_cast<uint32_t>(L::kPieces)) return false;
      publish();
    }
    if (((key0 - win) >> 4) + KS / 16 > 32) look_up();
    const int s = static_cast<int>(n_cp % NS);
    const uint32_t dst = ring + s * L::kStage + dst0;
#pragma unroll
    for (int g = 0; g < KS / 16; ++g) {
      const int64_t at = __shfl_sync(0xffffffffu, win_at, (((key0 - win) >> 4) + g) & 31);
      const int rows = at < 0 ? 0 : wk.k_hi - key0 - g * 16;  // of this run's 16
      const char* k = k0_ptr + (at < 0 ? 0 : 2 * at);
      // row g * 16 + i * kRows + c_row: its 16-byte chunks are permuted by the row's last bits
      if (rows >= 16) {
#pragma unroll
        for (int i = 0; i < 16 / kRows; ++i) {
          const uint32_t d = (dst + (g * 16 + i * kRows) * 128) ^ (((i * kRows) & 7) << 4);
          cp_async16(d, k);
          cp_async16(d + kVoff, k + v_minus_k);
          k += row_step;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < 16 / kRows; ++i) {
          const uint32_t d = (dst + (g * 16 + i * kRows) * 128) ^ (((i * kRows) & 7) << 4);
          const bool in = i * kRows + c_row < rows;
          const char* from = in ? k + i * row_step : reinterpret_cast<const char*>(a.kc);
          cp_async16_zfill(d, from, in ? 16 : 0);
          cp_async16_zfill(d + kVoff, in ? from + v_minus_k : from, in ? 16 : 0);
        }
      }
    }
    cp_async_arrive(full + s);
    ++n_cp;
    --left;
    key0 += KS;
    return true;
  };

  uint32_t n_it = 0, n_done = 0;  // tiles and pieces computed
  Piece p;                        // the one being computed, tile j of it next
  p.n_kt = 0;
  int j = 0;
  bool fresh = true, ok = true;
  uint32_t qf[NR][D / 16][2];
  int lim[NR][2];  // key limits of this thread's two statistics rows of each tile
  int lim_min = 0;  // the least of the tile's rows
  float o[NR][D / 16][4];
  float m[NR][2], lb[NR][2], lf[NR][2];
  // One turn: fill the ring, then a tile. (Each part stands in the code once: what a step runs for
  // the first time comes from L2 instruction by instruction, and a short step is mostly that.)
  while (true) {
#pragma unroll 1
    while (n_cp - n_it < static_cast<uint32_t>(NS) && copy_next(n_done)) {
    }
    if (fresh) {
      fresh = false;
      j = 0;
      p = pieces[n_done % L::kPieces];
      if (p.n_kt < 0) break;
      // Rows are found once, lane r row r, and handed on: the code of a step is short.
      const __nv_bfloat16* my_q = q_row(a, p, lane % MT);
      const int my_lim = row_limit(a, p, lane % MT);
      if (kSeveral) lim_min = __reduce_min_sync(0xffffffffu, my_q ? my_lim : p.keys);
      // B fragments of Q^T: row lane/4 of each tile, features (lane%4)*2 and +8 of each 16
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        const __nv_bfloat16* qp = shfl_ptr(my_q, c * 8 + (lane >> 2));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[c][k][e] = qp ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + e * 8 + (lane & 3) * 2) : 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          lim[c][e] = __shfl_sync(0xffffffffu, my_lim, c * 8 + (lane & 3) * 2 + e);
      }
#pragma unroll
      for (int c = 0; c < NR; ++c) {
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][n][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[c][e] = -INFINITY;
          lb[c][e] = lf[c][e] = 0.f;
        }
      }
    }
    if (j < p.n_kt) {
      const int s = static_cast<int>(n_it % NS);
      ok = __all_sync(0xffffffffu, mbar_wait(full + s, (n_it / NS) & 1));
      if (!ok) break;
      const uint32_t sk = ring + s * L::kStage, sv = sk + kVoff;
      const int k0 = j * KS;
      float sc[NR][KS / 16][4], sd[NR][KS / 16][4];  // two chains of sums: half the latency
#pragma unroll
      for (int c = 0; c < NR; ++c)
#pragma unroll
        for (int t = 0; t < KS / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[c][t][e] = sd[c][t][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int ch = (k & 3) * 2 + (lane >> 4);
#pragma unroll
        for (int t = 0; t < KS / 16; ++t) {
          const int r = t * 16 + (lane & 15);
          uint32_t ka[4];
          ldsm4(ka, sk + (k >> 2) * kHalf + r * 128 + ((ch ^ (r & 7)) << 4));
#pragma unroll
          for (int c = 0; c < NR; ++c)
            mma16816(k & 1 ? sd[c][t] : sc[c][t], ka, qf[c][k][0], qf[c][k][1]);
        }
      }
      // scores: [e] = key (lane/4) + 8 (e/2), row (lane%4)*2 + e%2 of the tile
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        float mx[2] = {m[c][0], m[c][1]};
#pragma unroll
        for (int t = 0; t < KS / 16; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool seen = k0 + t * 16 + (lane >> 2) + (e >> 1) * 8 < lim[c][e & 1];
            sc[c][t][e] = seen ? (sc[c][t][e] + sd[c][t][e]) * a.scale_log2 : -INFINITY;
            mx[e & 1] = fmaxf(mx[e & 1], sc[c][t][e]);
          }
        float al[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1)
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], x));
          base[e] = mx[e] == -INFINITY ? 0.f : mx[e];
          al[e] = ex2_approx(m[c][e] - base[e]);
        }
        if (__any_sync(0xffffffffu, mx[0] > m[c][0] || mx[1] > m[c][1])) {
#pragma unroll
          for (int n2 = 0; n2 < D / 16; ++n2)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][n2][e] *= al[e & 1];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            lb[c][e] *= al[e];
            lf[c][e] *= al[e];
            m[c][e] = mx[e];
          }
        }
        // weights, rounded to bf16 once for the product; two rows of one key are packed and
        // transposed into the product's B layout (two keys of one row)
#pragma unroll
        for (int t = 0; t < KS / 16; ++t) {
          uint32_t pb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = ex2_approx(sc[c][t][2 * e] - base[0]);
            const float p1 = ex2_approx(sc[c][t][2 * e + 1] - base[1]);
            lf[c][0] += p0;
            lf[c][1] += p1;
            const uint32_t w = pack_bf16(p0, p1);
            add_bf16x2(lb[c][0], lb[c][1], w);
            pb[e] = movmatrix(w);
          }
          sc[c][t][0] = __uint_as_float(pb[0]);
          sc[c][t][1] = __uint_as_float(pb[1]);
        }
      }
      if (kSeveral && min(k0 + KS, p.keys) > lim_min &&
          any_not_finite<D, KS>(sv, max(lim_min - k0, 0), lane)) {
#pragma unroll 1
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            uint32_t w = 0;  // the word of P^T that holds key k
#pragma unroll
            for (int x = 0; x < KS / 8; ++x)
              if (x == k >> 3) w = __float_as_uint(sc[c][x >> 1][x & 1]);
            float pk[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t u = __shfl_sync(0xffffffffu, w, ((lane & 3) * 2 + e) * 4 + ((k & 7) >> 1));
              pk[e] = __uint_as_float(k & 1 ? u & 0xffff0000u : u << 16);
            }
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              const float v = __uint_as_float(static_cast<uint32_t>(
                                  ld_shared_u16(v_at<KS>(sv, k, d * 8 + (lane >> 2)))) << 16);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (k0 + k < lim[c][e]) o[c][d >> 1][2 * (d & 1) + e] += pk[e] * v;
            }
          }
      } else {
#pragma unroll
        for (int t = 0; t < KS / 16; ++t)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const int r = t * 16 + ((lane >> 4) << 3) + (lane & 7);
            const int ch = (d & 3) * 2 + ((lane >> 3) & 1);
            uint32_t va[4];
            ldsm4_t(va, sv + (d >> 2) * kHalf + r * 128 + ((ch ^ (r & 7)) << 4));
#pragma unroll
            for (int c = 0; c < NR; ++c)
              mma16816(o[c][d], va, __float_as_uint(sc[c][t][0]), __float_as_uint(sc[c][t][1]));
          }
      }
      __syncwarp();
      ++n_it;
      if (++j < p.n_kt) continue;
    }
    // statistics over the lanes that share a row
#pragma unroll
    for (int c = 0; c < NR; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          lb[c][e] += __shfl_xor_sync(0xffffffffu, lb[c][e], x);
          lf[c][e] += __shfl_xor_sync(0xffffffffu, lf[c][e], x);
        }
    // row (lane%4)*2 + e of a tile: this lane has features lane/4 + 8 i of it
    RowOut mine = {nullptr, nullptr, nullptr, nullptr};
    if (p.row0 + lane % MT < p.n_rows) mine = row_out(a, p, lane % MT, MT, D, lane < MT);
    const bool sole = p.parts == 1 && a.prefix == 0;
    const int d0 = lane >> 2;
    if (sole) {
#pragma unroll
      for (int c = 0; c < NR; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          __nv_bfloat16* to = shfl_ptr(mine.o, c * 8 + (lane & 3) * 2 + e);
          float* to_lse = shfl_ptr(mine.lse, c * 8 + (lane & 3) * 2 + e);
          if (!to) continue;
          const float inv = lb[c][e] == 0.f ? 0.f : 1.f / lb[c][e];
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              to[n * 16 + f * 8 + d0] = __float2bfloat16_rn(o[c][n][2 * f + e] * inv);
          if (to_lse && d0 == 0) *to_lse = (m[c][e] + log2f(lf[c][e])) * 0.69314718055994530942f;
        }
    } else {
#pragma unroll
      for (int c = 0; c < NR; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* to = shfl_ptr(mine.part, c * 8 + (lane & 3) * 2 + e);
          float4* to_ml = shfl_ptr(mine.ml, c * 8 + (lane & 3) * 2 + e);
          if (!to) continue;
          if (lf[c][e] != 0.f) {  // NaN goes through
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
              for (int f = 0; f < 2; ++f) to[n * 16 + f * 8 + d0] = o[c][n][2 * f + e];
          }
          if (d0 == 0) *to_ml = make_float4(m[c][e], lb[c][e], lf[c][e], 0.f);
        }
    }
    ++n_done;
    fresh = true;
  }
  if (!ok) {  // a copy did not arrive within the limit
    if (lane == 0) atomicOr(a.err, kErrWaitTimeout | 0x10000u);
    for (uint32_t j = n_it; j < n_cp; ++j) mbar_wait(full + j % NS, (j / NS) & 1, 100000000ull);
  }
  // The join may start as blocks end (its own start in the middle of the work, waiting beside it,
  // cost 12 of 113 us over 131072 keys). The prefix kernel that this one may have started beside is
  // done before this one is, so that what follows this one follows both.
  launch_dependents();
  grid_dependency_wait();
}

// ---- more rows: one block a worker --------------------------------------------------------------
//
// Row tiles of 64: one producer warp, which walks the share, publishes each piece and streams its
// keys and values through a ring of 64-key stages, running ahead into the next pieces, and four
// consumer warps, each with 16 rows and every stage: S = Q K^T, O += P V. Bound: the consumers'
// time for a tile, 3400 to 3900 cycles with two blocks an SM (17 of the 23 bytes a cycle that HBM
// could bring). Warps without rows take part all the same: letting them skip their products made
// 20 to 40 rows 3 % slower.
constexpr int kThreads = 160;
constexpr int kPieces = 4;     // pieces published ahead

template <int D>
struct PLayout {
  static constexpr int kKeys = 64;
  static constexpr int kStage = 2 * kKeys * D * 2;  // K then V
  static constexpr int kStages = 98304 / kStage;
  static constexpr int kBar = kStages * kStage;
  static constexpr int kPiece = kBar + (2 * kStages + 2 * kPieces + 2) * 8;
  static constexpr int kAbort = kPiece + kPieces * static_cast<int>(sizeof(Piece));
  static constexpr int kBytes = kAbort + 16 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using L = PLayout<D>;
  constexpr int MT = 64;
  constexpr int KS = L::kKeys, NS = L::kStages;
  constexpr int kHalf = KS * 128;      // bytes of a stage's 64 features of K or V
  constexpr int kVoff = KS * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + NS;
  uint64_t* piece_full = empty + NS;
  uint64_t* piece_empty = piece_full + kPieces;
  uint64_t* meet = piece_empty + kPieces;  // the four consumer warps among themselves
  Piece* pieces = reinterpret_cast<Piece*>(smem + L::kPiece);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 128) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(piece_full + i, 1);
      mbar_init(piece_empty + i, 4);
    }
    mbar_init(meet, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

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
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int bx = a.box_rows;  // divides page_size and the stage's keys
    const int r = lane / (D / 64) * bx, half = lane % (D / 64);
    const bool mine = r < KS;
    const uint32_t off = half * kHalf + r * 128;
    Walk<KS, MT> wk;
    wk.init(a, lane, 0, 1, static_cast<uint32_t>(a.least),
            Walk<KS, MT>::begin(a, lane, blockIdx.x == 0));
    uint32_t n_it = 0, n_pc = 0;
    bool ok = true;
    while (ok) {
      Piece p;
      const bool more = wk.next(a, &p);
      if (!more) p.n_kt = -1;
      const int ps = n_pc % kPieces;
      if (n_pc >= kPieces) ok = __all_sync(0xffffffffu, wait(piece_empty + ps, (n_pc / kPieces - 1) & 1));
      if (!ok) break;
      if (lane == 0) {
        pieces[ps] = p;
        mbar_arrive(piece_full + ps);
      }
      ++n_pc;
      if (!more) break;
      const int32_t* pages = p.own ? a.table + wk.b * a.table_stride : a.ptable;
      for (int j = 0; j < p.n_kt; ++j, ++n_it) {
        const int s = static_cast<int>(n_it % NS);
        // A box past the keys, or of a page that does not exist, lies outside the tensor map
        // and reads as zeros; nothing outside the caches is touched.
        const int key = wk.k_lo + j * KS + r;
        int page = -1, slot = 0;
        if (mine && key < wk.k_hi) {
          const uint32_t pg = static_cast<uint32_t>(key) / static_cast<uint32_t>(a.page_size);
          page = pages[pg];
          slot = key - static_cast<int>(pg) * a.page_size;
          if (page < 0 || page >= a.n_pages) {
            page = -1;
            atomicOr(a.err, kErrBadPage);
          }
        }
        if (n_it >= NS) ok = __all_sync(0xffffffffu, wait(empty + s, (n_it / NS - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + s, L::kStage);
        __syncwarp();
        if (mine) {
          const uint32_t dst = smem_u32(smem) + s * L::kStage + off;
          tma_load_4d(dst, &tm_k, half * 64, slot, p.kvh, page, full + s);
          tma_load_4d(dst + kVoff, &tm_v, half * 64, slot, p.kvh, page, full + s);
        }
      }
    }
    if (!ok) {  // copies in flight land before the block's shared memory goes
      for (uint32_t j = (n_it >= NS ? n_it - NS : 0); j < n_it; ++j)
        mbar_wait(full + j % NS, (j / NS) & 1, 100000000ull);
    }
  } else {
    // ---------------- consumers ----------------
    {
      // the tables, on their way to L2 while the producer reads the lengths
      const uint32_t line = blockIdx.x * 128 + threadIdx.x;
      const uint32_t per = static_cast<uint32_t>(min((a.max_pages + 31) / 32, int64_t(1) << 20));
      const uint32_t b = line / per;
      if (b < static_cast<uint32_t>(a.B))
        prefetch_l2(a.table + b * a.table_stride + (line - b * per) * 32);
    }
    const uint32_t sm0 = smem_u32(smem);
    uint32_t n_it = 0, n_meet = 0, n_pc = 0;
    bool ok = true;
    // Every consumer warp has come here, and sees what the others wrote; false on expiry.
    auto meet_all = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      return __all_sync(0xffffffffu, wait(meet, n_meet++ & 1));
    };
    // Values past the piece's last key (slots of its last page that no token fills) may be
    // anything, infinities and NaN among them, and 0 * inf is not 0: rows [r0, r0 + n) of the
    // stage's V are cleared from row `valid` on.
    auto clear_v = [&](uint32_t sv, int r0, int n, int valid) {
      for (int x = lane; x < n * (D / 8); x += 32) {
        const int r = r0 + x / (D / 8), ch = x % (D / 8);
        if (r >= valid)
          st_shared_v4(sv + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
      }
      fence_proxy_async_smem();  // before TMA may fill the stage again
    };
    while (ok) {
      const int ps = n_pc % kPieces;
      ok = __all_sync(0xffffffffu, wait(piece_full + ps, (n_pc / kPieces) & 1));
      if (!ok) break;
      const Piece p = pieces[ps];
      __syncwarp();
      if (lane == 0) mbar_arrive(piece_empty + ps);
      ++n_pc;
      if (p.n_kt < 0) break;

      const int r_lo = lane >> 2;
      uint32_t qf[D / 16][4];
      int lim[2];
      const int my_row = warp * 16 + (lane & 15);  // found here once for the warp
      const __nv_bfloat16* my_q = q_row(a, p, my_row);
      const int my_lim = row_limit(a, p, my_row);
      const int lim_min = __reduce_min_sync(0xffffffffu, my_q ? my_lim : p.keys);
      const int lim_max = __reduce_max_sync(0xffffffffu, my_lim);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const __nv_bfloat16* qp = shfl_ptr(my_q, r_lo + 8 * e);
        lim[e] = __shfl_sync(0xffffffffu, my_lim, r_lo + 8 * e);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            qf[k][e + 2 * f] = qp ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + f * 8 + (lane & 3) * 2) : 0u;
      }
      float o[D / 8][4];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, lb[2] = {0.f, 0.f}, lf[2] = {0.f, 0.f};
      for (int j = 0; j < p.n_kt; ++j, ++n_it) {
        const int s = static_cast<int>(n_it % NS);
        ok = __all_sync(0xffffffffu, wait(full + s, (n_it / NS) & 1));
        if (!ok) break;
        const uint32_t sk = sm0 + s * L::kStage, sv = sk + kVoff;
        const int k0 = j * KS;
        if (k0 + KS > p.keys) {
          clear_v(sv, warp * 16, 16, p.keys - k0);
          ok = meet_all();
          if (!ok) break;
        }
        float sc[KS / 8][4];
#pragma unroll
        for (int n = 0; n < KS / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int ch = (k & 3) * 2 + ((lane >> 3) & 1);
#pragma unroll
          for (int kg = 0; kg < KS / 16; ++kg) {
            const int r = kg * 16 + ((lane >> 4) << 3) + (lane & 7);
            uint32_t kb[4];
            ldsm4(kb, sk + (k >> 2) * (kHalf) + r * 128 + ((ch ^ (r & 7)) << 4));
            mma16816(sc[2 * kg], qf[k], kb[0], kb[1]);
            mma16816(sc[2 * kg + 1], qf[k], kb[2], kb[3]);
          }
        }
        // scale, mask, running maximum
        const int kb0 = k0 + (lane & 3) * 2;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < KS / 8; ++n)
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
        uint32_t pf[KS / 16][4];
#pragma unroll
        for (int n = 0; n < KS / 8; ++n) {
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
        if (k0 >= lim_max) {
          // no row of the warp sees a key of the tile: no weights, and no values to look over (a first
          // chunk of 8192 tokens has half its tiles here)
        } else if (min(k0 + KS, p.keys) > lim_min &&
                   any_not_finite<D, KS>(sv, max(lim_min - k0, 0), lane)) {
#pragma unroll 1
          for (int k = 0; k < KS; ++k) {
            float pk[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w = 0;  // the word of P that holds key k
#pragma unroll
              for (int x = 0; x < KS / 8; ++x)
                if (x == k >> 3) w = pf[x >> 1][(x & 1) * 2 + e];
              w = __shfl_sync(0xffffffffu, w, (lane & ~3) | ((k & 7) >> 1));
              pk[e] = __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              const uint32_t v = ld_shared_u32(v_at<KS>(sv, k, n * 8 + (lane & 3) * 2));
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (k0 + k < lim[e]) {
                  o[n][2 * e] += pk[e] * __uint_as_float(v << 16);
                  o[n][2 * e + 1] += pk[e] * __uint_as_float(v & 0xffff0000u);
                }
            }
          }
        } else {
#pragma unroll
          for (int kg = 0; kg < KS / 16; ++kg)
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
              const int r = kg * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
              const int ch = (dp & 3) * 2 + (lane >> 4);
              uint32_t vb[4];
              ldsm4_t(vb, sv + (dp >> 2) * (kHalf) + r * 128 + ((ch ^ (r & 7)) << 4));
              mma16816(o[2 * dp], pf[kg], vb[0], vb[1]);
              mma16816(o[2 * dp + 1], pf[kg], vb[2], vb[3]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + s);
      }
      if (!ok) break;
      RowOut mine = {nullptr, nullptr, nullptr, nullptr};
      if (p.row0 + my_row < p.n_rows) mine = row_out(a, p, my_row, MT, D, lane < 16);
      const bool sole = p.parts == 1 && a.prefix == 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lb[e] += __shfl_xor_sync(0xffffffffu, lb[e], 1);
        lb[e] += __shfl_xor_sync(0xffffffffu, lb[e], 2);
        lf[e] += __shfl_xor_sync(0xffffffffu, lf[e], 1);
        lf[e] += __shfl_xor_sync(0xffffffffu, lf[e], 2);
        if (sole) {
          __nv_bfloat16* to = shfl_ptr(mine.o, r_lo + 8 * e);
          float* to_lse = shfl_ptr(mine.lse, r_lo + 8 * e);
          if (!to) continue;
          const float inv = lb[e] == 0.f ? 0.f : 1.f / lb[e];
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t*>(to + n * 8 + (lane & 3) * 2) =
                pack_bf16(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
          if (to_lse && (lane & 3) == 0) *to_lse = (m[e] + log2f(lf[e])) * 0.69314718055994530942f;
        } else {
          float* to = shfl_ptr(mine.part, r_lo + 8 * e);
          float4* to_ml = shfl_ptr(mine.ml, r_lo + 8 * e);
          if (!to) continue;
          if (lf[e] != 0.f) {  // NaN goes through
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(to + n * 8 + (lane & 3) * 2) =
                  make_float2(o[n][2 * e], o[n][2 * e + 1]);
          }
          if ((lane & 3) == 0) *to_ml = make_float4(m[e], lb[e], lf[e], 0.f);
        }
      }
    }
  }
  // The join may start as blocks end (its own start in the middle of the work, waiting beside it,
  // cost 12 of 113 us over 131072 keys). The prefix kernel that this one may have started beside is
  // done before this one is, so that what follows this one follows both.
  launch_dependents();
  grid_dependency_wait();
}

// Joins the parts of a row: kWarps warps per (row, head), warp u taking the parts u, u + kWarps, ...,
// their statistics 32 at a time (one a lane) with a running maximum, their numerators eight at a
// time; the warps' sums are joined in shared memory. The order of the sums is fixed. A row's parts
// are the prefix kernel's, then the pieces that desc names for the prefix and for its own keys.
// Bound: latency (dependent loads) for few rows, L2 for many. The prefix kernel's parts lie where the
// row says, so their statistics and the first eight numerators are asked for together with desc.
template <int D, int kWarps>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  constexpr int kRows = 8 / kWarps;  // rows per block
  constexpr int kQ = 8;              // numerators in flight per warp
  __shared__ float red[kWarps > 1 ? 8 : 1][D + 3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = warp % kWarps;
  const int64_t x = blockIdx.x * int64_t(kRows) + warp / kWarps;
  const int64_t t = div_fl(x, a.Hq);
  const int h = static_cast<int>(x - t * a.Hq);
  bool live = t < a.rows;
  if (live && a.cu) live = t < a.cu[a.B] && t >= a.cu[0];  // rows of no sequence stay as they are
  grid_dependency_wait();
  const int64_t step = a.rows * a.Hq;
  const int64_t at = t * a.Hq + h;
  const int n_x = live && a.splits_x ? a.splits_p : 0;
  int n_p = 0, n_o = 0;
  int64_t first_p = 0, first_o = 0;
  auto load = [&](const float* o, float (&r)[E]) {
    if (E == 4) {
      const float4 f = *reinterpret_cast<const float4*>(o + lane * E);
      r[0] = f.x; r[1] = f.y; r[E - 2] = f.z; r[E - 1] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(o + lane * E);
      r[0] = f.x; r[1] = f.y;
    }
  };
  int2 own = make_int2(0, 0), pre = make_int2(0, 0);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float r[kQ][E];
  if (live) {
    own = a.desc[step + at];
    if (a.prefix && !a.splits_x) pre = a.desc[at];
    if (lane * kWarps + u < n_x) v = a.part_ml[(lane * kWarps + u) * step + at];
#pragma unroll
    for (int q = 0; q < kQ; ++q)  // one that was not written (no keys) is passed over below
      if (q * kWarps + u < n_x) load(a.part_o + ((q * kWarps + u) * step + at) * D, r[q]);
    first_o = own.x;
    n_o = own.y;
    first_p = pre.x;
    n_p = pre.y;
    live = n_o != 0;  // finished by the kernel before
    // stay inside the slots whatever desc holds (cu_rows that decrease)
    const int64_t top = a.n_slots * a.mt;
    if (first_o < 0 || n_o < 0 || first_o + (n_o - int64_t(1)) * a.mt >= top) n_o = 0;
    if (first_p < 0 || n_p < 0 || first_p + (n_p - int64_t(1)) * a.mt >= top) n_p = 0;
  }
  if (kWarps == 1 && !live) return;
  const int parts = live ? n_x + n_p + n_o : 0;
  const int mine = parts > u ? (parts - u + kWarps - 1) / kWarps : 0;
  // row of statistics and numerators of this warp's i-th part
  auto where = [&](int i, const float4** ml, const float** o) {
    const int p = i * kWarps + u;
    if (p < n_x) {
      *ml = a.part_ml + p * step + at;
      *o = a.part_o + (p * step + at) * D;
    } else {
      const int64_t s = p < n_x + n_p ? first_p + static_cast<int64_t>(p - n_x) * a.mt
                                      : first_o + static_cast<int64_t>(p - n_x - n_p) * a.mt;
      *ml = a.slot_ml + s;
      *o = a.slot_o + s * D;
    }
  };
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float M = -INFINITY, lb = 0.f, lf = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const float4* ml;
    const float* o;
    if (i0 + lane < mine && (i0 || lane * kWarps + u >= n_x)) {
      where(i0 + lane, &ml, &o);
      v = *ml;
    }
    // lane i: the weight of part i0 + i; a part without keys (sum exactly 0) has written no
    // numerator and is passed over, one with NaN is not
    const bool has = i0 + lane < mine && v.z != 0.f;
    float top = has ? fmaxf(M, v.x) : M;
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    const float old = M == -INFINITY ? 0.f : ex2_approx(M - top);
    M = top;
    const float w = has ? ex2_approx(v.x - M) : -1.f;
    lb = lb * old + (has ? w * v.y : 0.f);
    lf = lf * old + (has ? w * v.z : 0.f);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll 1
    for (int q0 = 0; q0 < 32 && i0 + q0 < mine; q0 += kQ) {
      float wq[kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        wq[q] = __shfl_sync(0xffffffffu, w, q0 + q);
        const bool there = wq[q] >= 0.f || wq[q] != wq[q];
        if (there && (i0 + q0 || q * kWarps + u >= n_x)) {
          where(i0 + q0 + q, &ml, &o);
          load(o, r[q]);
        }
        if (!there) wq[q] = -1.f;
      }
#pragma unroll
      for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(wq[q] < 0.f)) acc[e] += wq[q] * r[q][e];
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) {
    lb += __shfl_xor_sync(0xffffffffu, lb, s);
    lf += __shfl_xor_sync(0xffffffffu, lf, s);
  }
  if (kWarps > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) red[warp % 8][lane * E + e] = acc[e];
    if (lane == 0) {
      red[warp % 8][D] = lb;
      red[warp % 8][D + 1] = lf;
      red[warp % 8][D + 2] = M;
    }
    __syncthreads();
    if (u != 0 || !live) return;
    lb = lf = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int v2 = 0; v2 < kWarps; ++v2) M = fmaxf(M, red[(warp + v2) % 8][D + 2]);
#pragma unroll
    for (int v2 = 0; v2 < kWarps; ++v2) {
      const float* rv = red[(warp + v2) % 8];
      const float w = rv[D + 2] == -INFINITY ? 0.f : ex2_approx(rv[D + 2] - M);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * rv[lane * E + e];
      lb += w * rv[D];
      lf += w * rv[D + 1];
    }
  }
  const float inv = lb == 0.f ? 0.f : 1.f / lb;  // no key in sight: zeros
  const int64_t bb = a.cu ? 0 : t / a.T, ii = a.cu ? t : t - bb * a.T;
  __nv_bfloat16* op = a.o + bb * a.o_b + ii * a.o_s + h * a.o_h + lane * E;
  if (E == 4)
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv),
                                               pack_bf16(acc[E - 2] * inv, acc[E - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(op) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (a.lse && lane == 0) {
    const int64_t li = a.cu ? h * a.rows + t : (bb * a.Hq + h) * a.T + ii;
    a.lse[li] = (M + log2f(lf)) * 0.69314718055994530942f;
  }
}

template <int D, int NR, bool kSeveral>
cudaError_t launch_decode_of(const PagedArgs& a, cudaStream_t stream) {
  using L = DLayout<D, NR>;
  const cudaError_t e = ensure_smem_attr(
      reinterpret_cast<const void*>(&paged_decode_kernel<D, NR, kSeveral>), L::kBytes);
  if (e != cudaSuccess) return e;
  // beside the prefix kernel, if there is one
  return launch_after(paged_decode_kernel<D, NR, kSeveral>, dim3(a.grid), dim3(kWarps * 32),
                      L::kBytes, stream, a.splits_x != 0, a);
}

template <int D, int NR>
cudaError_t launch_decode(const PagedArgs& a, cudaStream_t stream) {
  return a.cu || a.T > 1 ? launch_decode_of<D, NR, true>(a, stream)
                         : launch_decode_of<D, NR, false>(a, stream);
}

template <int D>
cudaError_t launch_rows(const PagedArgs& a, const CUtensorMap& km, const CUtensorMap& vm,
                        cudaStream_t stream) {
  using L = PLayout<D>;
  const cudaError_t e =
      ensure_smem_attr(reinterpret_cast<const void*>(&paged_rows_kernel<D>), L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(paged_rows_kernel<D>, dim3(a.grid), dim3(kThreads), L::kBytes, stream,
                      a.splits_x != 0, km, vm, a);
}

// Whether the prefix goes to the tensor-core kernel with its 128-row tiles, or to the kernels here
// together with the own keys, in tiles of 16 (or 64) rows that read it again from L2 each. The extra
// launch and the wider partial results cost about 5 us, so it takes rows x keys to pay (32 q-heads
// on 8 kv-heads, D 128, 200 own keys, one new token; us there / here):
//     rows a kv-head    32           64           128          256          512
//     prefix   512      18 / 15      19 / 16      21 / 16      25 / 22      35 / 34
//     prefix  2048      21 / 20      23 / 19      25 / 25      29 / 33      39 / 58
//     prefix  4096      22 / 20      25 / 26      28 / 32      32 / 50      43 / 92
//     prefix 16384      32 / 35      36 / 49      39 / 83      44 / 144     65 / 268
// (the same border with 16 heads of 64). With 64-row tiles the border lies higher: 128 rows on 4096
// keys 28 / 24, on 16384 39 / 49; 256 rows on 4096 31 / 37.
bool prefix_on_tc(const PagedArgs& a, int64_t rows_o) {
  const int64_t rows = a.rows * a.G;
  return a.prefix >= 128 && rows > 16 && rows * a.prefix >= (int64_t(1) << (rows_o > 16 ? 20 : 18));
}

}  // namespace

void plan_paged(PagedArgs* a, int64_t max_q, int64_t max_len) {
  if (max_len > 0x7fffffff) max_len = 0x7fffffff;  // lengths are 32-bit; a hint may be anything
  const int64_t rows_o = max_q * a->G, rows_p = a->rows * a->G;
  a->splits_x = a->splits_p = a->tiles_p = 0;
  if (prefix_on_tc(*a, rows_o)) {
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
  // a sequence's own rows choose the kernel; a prefix beside them takes several row tiles
  const int64_t most = a->prefix && !a->splits_x ? rows_p : rows_o;
  a->mt = rows_o > 16 ? 64 : most <= 8 ? 8 : 16;
  // segments: every sequence's rows fill whole tiles and one that is not full
  const int64_t segs = (rows_p / a->mt + a->B) * a->Hkv;
  const int64_t segs_p = a->prefix && !a->splits_x ? (rows_p + a->mt - 1) / a->mt * a->Hkv : 0;
  a->segs = segs;
  a->segs_p = segs_p;
  // Workers: eight warps on each SM, or two blocks; fewer where there are fewer shares. A share is
  // at least 32 keys of a decode step, so that no copy of a short one waits for a stage (64: 1.5 us
  // more of 11 on 300 keys of 128; the parts that it makes more cost the join 0.3).
  const bool warps = a->mt != 64;
  const int ks = a->ks = warps ? 2048 / a->D : 64;
  a->least = warps ? 32 / ks : 1;
  const int64_t t_o = (max_len + ks - 1) / ks, t_p = (a->prefix + ks - 1) / ks;
  const int64_t tiles = segs * t_o + segs_p * t_p;
  const int64_t want = (tiles + a->least - 1) / a->least, most_blocks = warps ? kSms : 2 * kSms;
  a->grid = static_cast<unsigned>(want < most_blocks ? want : most_blocks);
  const int64_t workers = static_cast<int64_t>(a->grid) * (warps ? kWarps : 1);
  a->n_slots = segs + segs_p + workers;
  // The join takes eight warps a row where rows are few and have many parts each (us of a step of
  // 32 q-heads on 8 kv-heads of 128, one warp / eight: 8 rows with 13 parts 18.5 / 16.5, 16 rows
  // with 34 parts 24.8 / 22.7; 24 rows with 5 parts 14.7 / 18.2).
  const int64_t all = segs * (kOver + t_o) + segs_p * (kOver + t_p);
  const int64_t share = all / workers > a->least ? all / workers : a->least;
  const int64_t parts = a->splits_p + (segs_p ? (kOver + t_p) / share + 1 : 0) + (kOver + t_o) / share + 1;
  a->wide = a->rows * a->Hq < 1024 && parts > 8;
}

cudaError_t launch_attn_paged(const PagedArgs& a, const CUtensorMap* k_map,
                              const CUtensorMap* v_map, cudaStream_t stream) {
  launch_begin(13, stream);
  cudaError_t e;
  if (a.D == 128)
    e = a.mt == 8    ? launch_decode<128, 1>(a, stream)
        : a.mt == 16 ? launch_decode<128, 2>(a, stream)
                     : launch_rows<128>(a, *k_map, *v_map, stream);
  else
    e = a.mt == 8    ? launch_decode<64, 1>(a, stream)
        : a.mt == 16 ? launch_decode<64, 2>(a, stream)
                     : launch_rows<64>(a, *k_map, *v_map, stream);
  launch_end(13, stream);
  return e;
}

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
  const int64_t rows = a.rows * a.Hq;
  const bool wide = a.wide;
  const int64_t blocks = wide ? rows : (rows + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 n(static_cast<unsigned>(blocks)), th(256);
  launch_begin(14, stream);
  cudaError_t e;
  if (a.D == 128)
    e = wide ? launch_after(paged_merge_kernel<128, 8>, n, th, 0, stream, true, a)
             : launch_after(paged_merge_kernel<128, 1>, n, th, 0, stream, true, a);
  else
    e = wide ? launch_after(paged_merge_kernel<64, 8>, n, th, 0, stream, true, a)
             : launch_after(paged_merge_kernel<64, 1>, n, th, 0, stream, true, a);
  launch_end(14, stream);
  return e;
}

}  // namespace upipe
