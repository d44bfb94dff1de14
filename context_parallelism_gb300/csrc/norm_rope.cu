// Norm of each head of q and k by its root mean square, and the rotation of its positions, in one
// pass: forward (also on the way into a paged cache) and backward.
//
// A head x of D features with weights w (or all ones), R the rotation of its position:
//   r = (mean x^2 + eps)^(-1/2),   y = R (w r x);
// the gradients for dy, with g = R^T dy (the rotation with the sine's sign turned), t = w g:
//   dx = r (t - x r^2 mean(t x)),   dw = sum over tokens and heads of g r x.
// Everything between the bf16 input and the one rounding of the output is fp32. r is recomputed in
// the backward, from an x that it reads anyway: nothing is kept from the forward.
//
// A thread owns the 16 features of a chunk (two 16-byte vectors, eight pairs) of a few heads of one
// token, and the 2, 4, 8, 16 or 32 lanes that share a head add up its sums by shuffles. Heads of one
// tensor form a thread's group; they share the angles and the weights. Whatever the layout, a chunk
// is held as the first features X of its eight pairs and the second ones Y, two to a register pair
// for the paired multiply-adds: in the half layout these are its two vectors, in the interleaved one
// the even and the odd elements of both.
//
// Bound: HBM, once enough bytes are in flight: the loads go to the thread's own places in shared
// memory as asynchronous copies, which hold no registers (131072 tokens of 32 + 8 heads of 128: 568 us
// with loads to registers, 385 so, 104 % of a copy's rate), and the angles are shared by eight heads.
// Copies past L1 want whole sectors to a request: with the 32 bytes of four interleaved pairs in one
// lane, two requests of half sectors, the backward of 8194 tokens took 123 us, now 83. The backward
// of 32768 tokens takes 173 us, 87 % of a copy's rate; its 325 instructions a lane and head are next.
#include "internal.h"
#include "rope.cuh"

namespace upipe {
namespace {

constexpr int kFwdThreads = 64;
constexpr int kFwdShort = 2, kFwdLong = 8;  // heads of one token per thread
constexpr int kBwdThreads = 128;
constexpr int kBwdShort = 2, kBwdLong = 8;
constexpr int kBwdAhead = 2;  // heads whose loads a thread has in flight

// Waits until all but the thread's last n groups of asynchronous copies have landed.
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Eight floats as four pairs.
struct F8 {
  uint64_t p[4];
};

// A chunk's vectors as the firsts X and seconds Y of its pairs, and back.
template <bool kInter>
__device__ __forceinline__ void unpack_chunk(const uint4& a, const uint4& b, F8& x, F8& y) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInter) {
      x.p[i] = f2_pack_u(w[2 * i] << 16, w[2 * i + 1] << 16);
      y.p[i] = f2_pack_u(w[2 * i] & 0xffff0000u, w[2 * i + 1] & 0xffff0000u);
    } else {
      x.p[i] = f2_pack_u(w[i] << 16, w[i] & 0xffff0000u);
      y.p[i] = f2_pack_u(w[4 + i] << 16, w[4 + i] & 0xffff0000u);
    }
  }
}

template <bool kInter>
__device__ __forceinline__ void pack_chunk(const F8& x, const F8& y, uint4& a, uint4& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, x1, y0, y1;
    f2_unpack(x.p[i], x0, x1);
    f2_unpack(y.p[i], y0, y1);
    if (kInter) {
      w[2 * i] = pack_bf16(x0, y0);
      w[2 * i + 1] = pack_bf16(x1, y1);
    } else {
      w[i] = pack_bf16(x0, x1);
      w[4 + i] = pack_bf16(y0, y1);
    }
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// The two vectors of a head that chunk c holds (D: none). Neighbouring lanes hold neighbouring vectors,
// whole sectors of a head to a request, in both layouts: 8 c and rot / 2 + 8 c of the rotated part,
// the first and the second half of the vectors behind it likewise.
__device__ __forceinline__ bool chunk_vectors(int c, int rot, int D, int* o0, int* o1) {
  const int nr = rot >> 4, nt = (D - rot + 15) >> 4, k = c - nr;
  if (k < 0) {
    *o0 = 8 * c;
    *o1 = rot / 2 + 8 * c;
    return true;
  }
  *o0 = k < nt ? rot + 8 * k : D;
  *o1 = k < nt ? rot + 8 * (nt + k) : D;
  return false;
}

// Feature of the head that X's (second = 0) or Y's i-th element is.
template <bool kInter>
__device__ __forceinline__ int feature(int i, int second, int o0, int o1) {
  if (kInter) return (i < 4 ? o0 + 2 * i : o1 + 2 * (i - 4)) + second;
  return (second ? o1 : o0) + i;
}

// Eight effective weights, offset + w or ones, from feature o on; zeros behind the head.
__device__ __forceinline__ void load_weights8(const NormArgs& a, int t, int o, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (o >= a.r.D) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  } else if (a.w[t]) {
    if (a.wide) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.w[t]) + o);
      const float4 u = p[0], v = p[1];
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    } else {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w[t]) + o), w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] += a.offset;
  }
}

// Those of a chunk's X and Y.
template <bool kInter>
__device__ __forceinline__ void load_weights(const NormArgs& a, int t, int o0, int o1, F8& x, F8& y) {
  float u[8], v[8];
  load_weights8(a, t, o0, u);
  load_weights8(a, t, o1, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kInter) {
      const float* w = i < 2 ? u : v;
      const int k = 4 * (i & 1);
      x.p[i] = f2_pack(w[k], w[k + 2]);
      y.p[i] = f2_pack(w[k + 1], w[k + 3]);
    } else {
      x.p[i] = f2_pack(u[2 * i], u[2 * i + 1]);
      y.p[i] = f2_pack(v[2 * i], v[2 * i + 1]);
    }
  }
}

__device__ __forceinline__ uint64_t both(float v) { return f2_pack(v, v); }

// Cosines and sines, times their factors, of chunk c's eight pairs at position pos. The fraction of a turn,
// p * phase modulo 2^64 (see rope.cu), is kept to 32 bits (2^-32 of a turn); its upper bits name the
// nearest quarter turn, and for the rest, x within pi / 4, the Taylor series up to x^9 and x^10 are
// off by less than 2^-28. About 20 instructions an angle, well under a general sine and cosine.
template <bool kInter>
__device__ __forceinline__ void chunk_turns(const RopeArgs& a, int c, int64_t pos, F8& cs, F8& sn) {
  const ulonglong2* ph = reinterpret_cast<const ulonglong2*>(a.phase) + (kInter ? 2 : 4) * c;
  const float m = a.mscale, ms = a.sin_scale;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 f = ph[kInter && i >= 2 ? a.rot / 8 + i - 2 : i];
    const uint32_t t0 = static_cast<uint32_t>((static_cast<uint64_t>(pos) * f.x) >> 32);
    const uint32_t t1 = static_cast<uint32_t>((static_cast<uint64_t>(pos) * f.y) >> 32);
    const uint32_t q0 = (t0 + 0x20000000u) >> 30, q1 = (t1 + 0x20000000u) >> 30;
    const float r0 = static_cast<float>(static_cast<int32_t>(t0 - (q0 << 30)));
    const float r1 = static_cast<float>(static_cast<int32_t>(t1 - (q1 << 30)));
    const uint64_t x = fmul2(f2_pack(r0, r1), both(6.283185307179586f * 0x1p-32f));
    const uint64_t z = fmul2(x, x);
    uint64_t s = ffma2(z, both(1.f / 362880), both(-1.f / 5040));
    s = ffma2(z, s, both(1.f / 120));
    s = ffma2(z, s, both(-1.f / 6));
    s = ffma2(fmul2(z, x), s, x);
    uint64_t d = ffma2(z, both(-1.f / 3628800), both(1.f / 40320));
    d = ffma2(z, d, both(-1.f / 720));
    d = ffma2(z, d, both(1.f / 24));
    d = ffma2(z, d, both(-0.5f));
    d = ffma2(z, d, both(1.f));
    float s0, s1, d0, d1;
    f2_unpack(s, s0, s1);
    f2_unpack(d, d0, d1);
    // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    const float a0 = q0 & 1 ? s0 : d0, b0 = q0 & 1 ? d0 : s0;
    const float a1 = q1 & 1 ? s1 : d1, b1 = q1 & 1 ? d1 : s1;
    const uint32_t n0 = ((q0 + 1) << 30) & 0x80000000u, n1 = ((q1 + 1) << 30) & 0x80000000u;
    const uint32_t k0 = (q0 << 30) & 0x80000000u, k1 = (q1 << 30) & 0x80000000u;
    cs.p[i] = fmul2(f2_pack_u(__float_as_uint(a0) ^ n0, __float_as_uint(a1) ^ n1), both(m));
    sn.p[i] = fmul2(f2_pack_u(__float_as_uint(b0) ^ k0, __float_as_uint(b1) ^ k1), both(ms));
  }
}

// <x, u> + <y, v>
__device__ __forceinline__ float dot_pairs(const F8& x, const F8& u, const F8& y, const F8& v) {
  uint64_t s = fmul2(x.p[0], u.p[0]), t = fmul2(y.p[0], v.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = ffma2(x.p[i], u.p[i], s);
    t = ffma2(y.p[i], v.p[i], t);
  }
  float lo, hi;
  f2_unpack(fadd2(s, t), lo, hi);
  return lo + hi;
}

// Sum over the lanes that share a head.
__device__ __forceinline__ float head_sum(float s, int lanes) {
  for (int m = lanes >> 1; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}

// (ss / D + eps)^(-1/2) of a head whose squares sum to ss. Heads whose squares leave the range in which
// fp32 keeps its digits are scaled by a power of two and summed again: down beside a mean above 2^117, up
// (kTiny) below 2^-96. The factor of the latter may be beyond fp32 itself: x and y become kLow times what
// they were and the result, that of these, is negative like kLow, which marks it. An eps of 2^-96 or more
// leaves no such head, so there are kernels without them: the path costs the backward registers (32768
// tokens 194 us with it, 175 without; half of each head interleaved, 8194 tokens: 98 and 84) and the
// forward 1 % (8194 tokens 57.7 and 57.1). All lanes of a warp call.
constexpr float kLow = -0x1p96f, kLeast = 0x1p-96f;
template <bool kTiny>
__device__ __forceinline__ float inverse_rms(const NormArgs& a, float ss, F8& x, F8& y) {
  const float t = fmaf(ss, a.inv_d, a.eps);
  float r = rsqrtf(t);
  const bool high = !(t <= 0x1p117f), low = kTiny && t < kLeast;
  if (__any_sync(0xffffffffu, high || low)) {
    const uint64_t c = both(kTiny && low ? kLow : 0x1p-96f);  // (not used for the others' heads)
    F8 u, v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u.p[i] = fmul2(x.p[i], c);
      v.p[i] = fmul2(y.p[i], c);
    }
    const float s = head_sum(dot_pairs(u, u, v, v), a.lanes);
    if (high) r = 0x1p-96f * rsqrtf(fmaf(s, a.inv_d, a.eps_down));
    if (kTiny) {
      const uint64_t k = both(low ? kLow : 1.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x.p[i] = fmul2(x.p[i], k);
        y.p[i] = fmul2(y.p[i], k);
      }
      if (low) r = -rsqrtf(fmaf(s, a.inv_d, a.eps_up));
    }
  }
  return r;
}

// f(0), .. f(n - 1) with the number a constant.
template <int n, int j = 0, typename F>
__device__ __forceinline__ void unrolled(F& f) {
  if constexpr (j < n) {
    f(std::integral_constant<int, j>());
    unrolled<n, j + 1>(f);
  }
}

// Thread -> (token, head group, lane of a head), lane fastest; groups number q's, k's, v's heads. A
// group's kPer heads share the angles and the weights, folded into one map of the chunk; all their
// loads are started before anything else.
template <bool kInter, bool kAppend, int kPer, bool kTiny>
__global__ void __launch_bounds__(kFwdThreads, 8) norm_rope_kernel(const NormArgs a) {
  __shared__ uint4 stage[2 * kPer][kFwdThreads];
  const RopeArgs& ra = a.r;
  const uint32_t idx = blockIdx.x * static_cast<uint32_t>(kFwdThreads) + threadIdx.x;
  const uint32_t item = idx >> a.log_lanes;
  const int c = static_cast<int>(idx & (a.lanes - 1));
  const uint32_t tok32 = item / ra.n_groups;
  int g = static_cast<int>(item - tok32 * ra.n_groups);
  // threads without work stay for the shuffles
  bool live = idx < ra.units;
  TokenPlace at{};
  live = live && place_token<kAppend>(ra, ra.tok0 + tok32, c == 0 && g == 0, &at);

  int t = 0;
  while (t < 2 && g >= a.groups[t]) g -= a.groups[t++];
  int o0, o1;
  const bool turns = chunk_vectors(c, ra.rot, ra.D, &o0, &o1);
  const bool two = o1 < ra.D;
  const bool cached = kAppend && t > 0, normed = t < 2;
  live = live && o0 < ra.D && !(cached && at.slot < 0);
  const int step = a.groups[t];
  const int mine = live ? (ra.heads[t] - g + step - 1) / step : 0;  // heads of this thread

  {
    const uint32_t to = smem_u32(&stage[0][threadIdx.x]);
    constexpr uint32_t kRow = kFwdThreads * 16;
    const __nv_bfloat16* src = ra.src[t] + at.b * ra.src_b[t] + at.i * ra.src_s[t] + g * ra.src_h[t];
    const int64_t src_step = step * ra.src_h[t];
#pragma unroll
    for (int j = 0; j < kPer; ++j, src += src_step) {
      if (j < mine) {
        cp_async16(to + 2 * j * kRow, src + o0);
        if (two) cp_async16(to + (2 * j + 1) * kRow, src + o1);
      }
      cp_async_commit();
    }
  }
  // X' = X ax + Y bx, Y' = Y ay + X by
  F8 ax{}, ay{}, bx{}, by{};
  if (live && normed) {
    load_weights<kInter>(a, t, o0, o1, ax, ay);
    if (turns) {
      F8 cs, sn;
      chunk_turns<kInter>(ra, c, at.pos, cs, sn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bx.p[i] = fmul2(fmul2(sn.p[i], ay.p[i]), both(-1.f));
        by.p[i] = fmul2(sn.p[i], ax.p[i]);
        ax.p[i] = fmul2(cs.p[i], ax.p[i]);
        ay.p[i] = fmul2(cs.p[i], ay.p[i]);
      }
    }
  }
  const int64_t dst_h = cached ? ra.head_stride : ra.dst_h[t];
  __nv_bfloat16* dst = ra.dst[t] + (cached ? at.slot : at.b * ra.dst_b[t] + at.i * ra.dst_s[t]) +
                       g * dst_h;
  auto head = [&](auto J) {
    constexpr int j = decltype(J)::value;
    cp_async_wait<kPer - 1 - j>();
    const bool here = j < mine;
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    if (here) {
      va = stage[2 * j][threadIdx.x];
      if (two) vb = stage[2 * j + 1][threadIdx.x];
    }
    F8 x, y;
    unpack_chunk<kInter>(va, vb, x, y);
    const float ss = head_sum(dot_pairs(x, x, y, y), a.lanes);
    const float r = inverse_rms<kTiny>(a, normed ? ss : 1.f, x, y);
    if (here) {
      if (normed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // r first: a head's features may leave fp32's range times the weights, its normed ones not
          const uint64_t u = fmul2(x.p[i], both(r)), v = fmul2(y.p[i], both(r));
          x.p[i] = fmul2(u, ax.p[i]);
          y.p[i] = fmul2(v, ay.p[i]);
          if (turns) {
            x.p[i] = ffma2(v, bx.p[i], x.p[i]);
            y.p[i] = ffma2(u, by.p[i], y.p[i]);
          }
        }
        pack_chunk<kInter>(x, y, va, vb);
      }
      *reinterpret_cast<uint4*>(dst + o0) = va;
      if (two) *reinterpret_cast<uint4*>(dst + o1) = vb;
    }
    dst += step * dst_h;
  };
  unrolled<kPer>(head);
}

// A set of `lanes` lanes keeps one head group and walks the tokens, so that its 16 sums of dw and its
// weights stay in registers; a block adds its sets' sums in order and leaves 2 D partial sums.
template <bool kInter, int kPer, bool kTiny>
__global__ void __launch_bounds__(kBwdThreads, 4) norm_rope_bwd_kernel(const NormArgs a) {
  static_assert(kPer % kBwdAhead == 0, "a head's slot is a constant");
  const RopeArgs& ra = a.r;
  // [slot][x: two vectors, dy: two][thread]; at the end the partial sums
  __shared__ uint4 ring[kBwdAhead * 4][kBwdThreads];
  const int sets = kBwdThreads >> a.log_lanes;
  const int set_in = static_cast<int>(threadIdx.x) >> a.log_lanes;
  const int c = static_cast<int>(threadIdx.x) & (a.lanes - 1);
  const uint32_t set = blockIdx.x * static_cast<uint32_t>(sets) + set_in;
  const uint32_t walkers = (gridDim.x * static_cast<uint32_t>(sets)) / ra.n_groups;
  const uint32_t walker = set / ra.n_groups;
  int g = static_cast<int>(set - walker * ra.n_groups);
  int t = 0;
  if (g >= a.groups[0]) {
    g -= a.groups[0];
    t = 1;
  }
  int o0, o1;
  const bool turns = chunk_vectors(c, ra.rot, ra.D, &o0, &o1);
  const bool in0 = o0 < ra.D, two = o1 < ra.D;
  const int step = a.groups[t];
  const int own = walker < walkers && in0 ? (ra.heads[t] - g + step - 1) / step : 0;
  F8 wx, wy, dwx{}, dwy{};
  load_weights<kInter>(a, t, o0, o1, wx, wy);

  const uint32_t to = smem_u32(&ring[0][threadIdx.x]);
  constexpr uint32_t kRow = kBwdThreads * 16;
  // the token that loads are started for, one ahead of the other in time
  struct Token {
    __nv_bfloat16* dx;
    int64_t pos;
    int heads;
  };
  const __nv_bfloat16 *px = nullptr, *pg = nullptr;
  auto enter = [&](int64_t token) {
    Token w{nullptr, 0, 0};
    if (own && token < a.tokens) {
      const int64_t b = ra.B == 1 ? 0 : div_fl(token, ra.S), i = token - b * ra.S;
      px = a.x[t] + b * a.x_b[t] + i * a.x_s[t] + g * a.x_h[t];
      pg = ra.src[t] + b * ra.src_b[t] + i * ra.src_s[t] + g * ra.src_h[t];
      w.dx = ra.dst[t] + b * ra.dst_b[t] + i * ra.dst_s[t] + g * ra.dst_h[t];
      w.pos = ra.pos ? ra.pos[token] : ra.pos0 + i;
      w.heads = own;
    }
    return w;
  };
  auto start = [&](bool is, int slot) {
    if (is) {
      cp_async16(to + slot * 4 * kRow, px + o0);
      cp_async16(to + (slot * 4 + 2) * kRow, pg + o0);
      if (two) {
        cp_async16(to + (slot * 4 + 1) * kRow, px + o1);
        cp_async16(to + (slot * 4 + 3) * kRow, pg + o1);
      }
    }
    cp_async_commit();
    px += step * a.x_h[t];
    pg += step * ra.src_h[t];
  };

  Token w = enter(walker);
#pragma unroll
  for (int j = 0; j < kBwdAhead; ++j) start(j < w.heads, j);

  // every lane of a warp takes the same number of steps: the shuffles want them all
  const int64_t tokens = (a.tokens + walkers - 1) / walkers;
  for (int64_t n = 0; n < tokens; ++n) {
    F8 cs{}, sn{};
    if (w.heads && turns) chunk_turns<kInter>(ra, c, w.pos, cs, sn);
    Token next{nullptr, 0, 0};
    auto head = [&](auto J) {
      constexpr int j = decltype(J)::value, slot = j % kBwdAhead, then = j + kBwdAhead;
      const bool here = j < w.heads;
      cp_async_wait<kBwdAhead - 1>();
      uint4 xa = make_uint4(0, 0, 0, 0), xb = xa, ga = xa, gb = xa;
      if (here) {
        xa = ring[slot * 4][threadIdx.x];
        ga = ring[slot * 4 + 2][threadIdx.x];
        if (two) {
          xb = ring[slot * 4 + 1][threadIdx.x];
          gb = ring[slot * 4 + 3][threadIdx.x];
        }
      }
      F8 x, y, u, v;
      unpack_chunk<kInter>(xa, xb, x, y);
      unpack_chunk<kInter>(ga, gb, u, v);
      if (then == kPer) next = enter((n + 1) * walkers + walker);
      start(then < kPer ? then < w.heads : then - kPer < next.heads, slot);
      const float ss = head_sum(dot_pairs(x, x, y, y), a.lanes);
      float r = inverse_rms<kTiny>(a, ss, x, y);
      if (!here) r = 0.f;  // without eps the zeros of no head would make dw NaN
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (turns) {
          const uint64_t p = u.p[i], q = v.p[i];
          u.p[i] = ffma2(p, cs.p[i], fmul2(fmul2(q, both(-1.f)), sn.p[i]));
          v.p[i] = ffma2(q, cs.p[i], fmul2(p, sn.p[i]));
        }
        x.p[i] = fmul2(x.p[i], both(r));
        y.p[i] = fmul2(y.p[i], both(r));
        dwx.p[i] = ffma2(u.p[i], x.p[i], dwx.p[i]);
        dwy.p[i] = ffma2(v.p[i], y.p[i], dwy.p[i]);
        u.p[i] = fmul2(u.p[i], wx.p[i]);
        v.p[i] = fmul2(v.p[i], wy.p[i]);
      }
      const float tx = head_sum(dot_pairs(u, x, v, y), a.lanes) * -a.inv_d;
      if (here) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u.p[i] = fmul2(both(r), ffma2(x.p[i], both(tx), u.p[i]));
          v.p[i] = fmul2(both(r), ffma2(y.p[i], both(tx), v.p[i]));
          if (kTiny && r < 0.f) {
            u.p[i] = fmul2(u.p[i], both(kLow));
            v.p[i] = fmul2(v.p[i], both(kLow));
          }
        }
        pack_chunk<kInter>(u, v, ga, gb);
        __nv_bfloat16* dx = w.dx + j * step * ra.dst_h[t];
        *reinterpret_cast<uint4*>(dx + o0) = ga;
        if (two) *reinterpret_cast<uint4*>(dx + o1) = gb;
      }
    };
    unrolled<kPer>(head);
    w = next;
  }
  cp_async_wait<0>();

  if (!a.part) return;
  // part[set][feature of the head]; a set's tensor follows from its group
  float* part = reinterpret_cast<float*>(&ring[0][0]);
  static_assert(sizeof(ring) >= kBwdThreads * 16 * 4, "the partial sums fit the ring");
  const int row = a.lanes * 16;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float lo, hi;
      f2_unpack(k ? dwy.p[i] : dwx.p[i], lo, hi);
      const int f = feature<kInter>(2 * i, k, o0, o1), h = feature<kInter>(2 * i + 1, k, o0, o1);
      if (f < ra.D) part[set_in * row + f] = lo;
      if (h < ra.D) part[set_in * row + h] = hi;
    }
  }
  __syncthreads();
  for (int f = threadIdx.x; f < 2 * ra.D; f += kBwdThreads) {
    const int which = f >= ra.D;
    float s = 0.f;
    for (int k = 0; k < sets; ++k) {
      const uint32_t gk = (blockIdx.x * static_cast<uint32_t>(sets) + k) % ra.n_groups;
      if ((gk >= static_cast<uint32_t>(a.groups[0])) == which) s += part[k * row + f - which * ra.D];
    }
    a.part[static_cast<int64_t>(blockIdx.x) * 2 * ra.D + f] = s;
  }
}

// dw[f] = the blocks' partial sums of feature f, in order within 32 interleaved runs.
constexpr int kRuns = 32;
__global__ void __launch_bounds__(32 * kRuns) norm_weights_kernel(const float* part, int blocks,
                                                                  int D, float* dq_w, float* dk_w) {
  __shared__ float run[kRuns][33];
  const int lane = threadIdx.x & 31, k0 = threadIdx.x >> 5, f = blockIdx.x * 32 + lane;
  grid_dependency_wait();
  float s = 0.f;
  if (f < 2 * D) {
#pragma unroll 8
    for (int k = k0; k < blocks; k += kRuns) s += part[static_cast<int64_t>(k) * 2 * D + f];
  }
  run[k0][lane] = s;
  __syncthreads();
  // a warp adds a feature's runs
  s = run[lane][k0];
#pragma unroll
  for (int m = kRuns / 2; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  const int g = blockIdx.x * 32 + k0;
  if (lane || g >= 2 * D) return;
  float* out = g < D ? dq_w : dk_w;
  if (out) out[g < D ? g : g - D] = s;
}

// Lanes per head, groups of up to `heads` heads.
void plan_groups(NormArgs* a, int heads) {
  a->per = heads;
  const int chunks = (a->r.D + 15) / 16;
  a->lanes = 1;
  a->log_lanes = 0;
  while (a->lanes < chunks) {
    a->lanes *= 2;
    ++a->log_lanes;
  }
  a->inv_d = 1.f / static_cast<float>(a->r.D);
  a->r.n_groups = 0;
  for (int t = 0; t < 3; ++t) {
    a->groups[t] = (a->r.heads[t] + heads - 1) / heads;
    a->r.n_groups += static_cast<uint32_t>(a->groups[t]);
  }
}

// Heads of a group in the backward: two in short calls (240 tokens of 32 + 8 heads of 128: 8.3 us, 10.8
// with eight), else eight (512 tokens: 12.1, 12.9 with two).
int bwd_heads(int64_t tokens, int heads, int D) {
  return tokens * heads * ((D + 15) / 16) < 152 * 1024 ? kBwdShort : kBwdLong;
}

template <bool kTiny, bool kAppend>
auto* fwd_kernel(int per, bool interleaved) {
  return per == kFwdLong ? interleaved ? norm_rope_kernel<true, kAppend, kFwdLong, kTiny>
                                       : norm_rope_kernel<false, kAppend, kFwdLong, kTiny>
                         : interleaved ? norm_rope_kernel<true, kAppend, kFwdShort, kTiny>
                                       : norm_rope_kernel<false, kAppend, kFwdShort, kTiny>;
}

template <bool kTiny>
auto* bwd_kernel(int per, bool interleaved) {
  return per == kBwdLong ? interleaved ? norm_rope_bwd_kernel<true, kBwdLong, kTiny>
                                       : norm_rope_bwd_kernel<false, kBwdLong, kTiny>
                         : interleaved ? norm_rope_bwd_kernel<true, kBwdShort, kTiny>
                                       : norm_rope_bwd_kernel<false, kBwdShort, kTiny>;
}

}  // namespace

cudaError_t launch_norm_rope(NormArgs a, bool interleaved, bool append, int64_t tokens,
                             cudaStream_t stream) {
  const int64_t H = a.r.heads[0] + a.r.heads[1] + a.r.heads[2];
  // two heads a thread while that leaves the SMs room (512 tokens of 32 + 8 heads of 128: 4.8 us, 5.5 with
  // eight), eight beyond (1024 tokens: 6.4, 7.4 with two)
  plan_groups(&a, tokens * H * ((a.r.D + 15) / 16) < 152 * 1536 ? kFwdShort : kFwdLong);
  const int64_t per_tok = static_cast<int64_t>(a.lanes) * a.r.n_groups;
  const bool tiny = a.eps < kLeast;
  auto* kernel = append ? tiny ? fwd_kernel<true, true>(a.per, interleaved) : fwd_kernel<false, true>(a.per, interleaved)
                 : tiny ? fwd_kernel<true, false>(a.per, interleaved)
                        : fwd_kernel<false, false>(a.per, interleaved);
  // thread indices fit 32 bits; a longer call goes in several launches
  const int64_t most = ((int64_t(1) << 31) - 1) / per_tok;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t n = tokens - t0 < most ? tokens - t0 : most;
    a.r.tok0 = t0;
    a.r.units = static_cast<uint32_t>(n * per_tok);
    const unsigned grid = static_cast<unsigned>((n * per_tok + kFwdThreads - 1) / kFwdThreads);
    launch_begin(16, stream);
    kernel<<<grid, kFwdThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    launch_end(16, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int norm_bwd_blocks(int64_t tokens, int D, int heads_q, int heads_k) {
  NormArgs a{};
  a.r.D = D;
  a.r.heads[0] = heads_q;
  a.r.heads[1] = heads_k;
  plan_groups(&a, bwd_heads(tokens, heads_q + heads_k, D));
  // a block for every block's worth of work, at most kNormBwdBlocks; at least a walker for each group
  const int sets = kBwdThreads / a.lanes;
  const int64_t least = (static_cast<int64_t>(a.r.n_groups) + sets - 1) / sets;
  const int64_t work = tokens > (int64_t(1) << 32) ? int64_t(1) << 40 : tokens * a.r.n_groups;
  int64_t b = (work + sets - 1) / sets;
  if (b > kNormBwdBlocks) b = kNormBwdBlocks;
  return static_cast<int>(b < least ? least : b);
}

cudaError_t launch_norm_rope_bwd(NormArgs a, bool interleaved, float* dq_w, float* dk_w,
                                 cudaStream_t stream) {
  plan_groups(&a, bwd_heads(a.tokens, a.r.heads[0] + a.r.heads[1], a.r.D));
  const int blocks = norm_bwd_blocks(a.tokens, a.r.D, a.r.heads[0], a.r.heads[1]);
  auto* kernel = a.eps < kLeast ? bwd_kernel<true>(a.per, interleaved) : bwd_kernel<false>(a.per, interleaved);
  launch_begin(16, stream);
  kernel<<<blocks, kBwdThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  launch_end(16, stream);
  if (e != cudaSuccess || !a.part) return e;
  launch_begin(16, stream);
  e = launch_after(norm_weights_kernel, dim3((2 * a.r.D + 31) / 32), dim3(32 * kRuns), 0, stream, true,
                   static_cast<const float*>(a.part), blocks, a.r.D, dq_w, dk_w);
  launch_end(16, stream);
  return e;
}

}  // namespace upipe
