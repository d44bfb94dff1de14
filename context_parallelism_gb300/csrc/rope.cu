// Rotary positions, and the append to a paged key/value cache that rotates on the way.
//
// Pair (x1, x2) of a head at position p with frequency f (radians a position):
//   y1 = m (x1 cos(p f) - x2 sin(p f)),   y2 = m (x2 cos(p f) + x1 sin(p f));
// the gradient is the transpose, the same map with the sine's sign turned. Pairs are
// (x_i, x_{i + rot/2}) in the half layout, (x_{2i}, x_{2i+1}) in the interleaved one.
//
// Angles. f is kept as a 64-bit fixed-point fraction of a turn, phase = round(f / (2 pi) 2^64),
// so p * phase modulo 2^64 is the fractional turn of the angle, exactly, for every 64-bit
// position: one integer multiply instead of a 64-bit floating-point range reduction or a table
// over positions. Read as a signed number it is the angle in half turns times 2^63, which
// sincospif takes without further reduction. The phase's own rounding (within 2^-64 of a turn:
// upipe_rope_phases divides in two doubles) reaches 2^-25 of a turn, a float's resolution, only at
// position 2^39.
//
// Bound: HBM. Each element is read and written once (4 bytes); a thread owns 8 frequencies (two
// 16-byte vectors of a head) and applies them to kHeads heads of one token, so the eight
// sincospif are shared by 64 elements. Measured: 131072 tokens of 32 + 8 heads of 128 (2.7 GB) in
// 387 us, 6.9 TB/s (2 heads a thread 464 us, 6 heads 410); 8192 tokens 30.8 us, of which the ramp
// is 5. Blocks of 64 threads end and start evenly: 256 cost 3 %. Streaming loads and stores changed
// nothing.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace upipe {
namespace {

constexpr int kThreads = 64;
constexpr int kHeads = 4;  // heads of one token per thread

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// Two vectors a, b of one head that hold eight pairs: (a_i, b_i) in the half layout,
// consecutive elements of a and then of b in the interleaved one.
template <bool kInter>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float (&c)[8],
                                       const float (&s)[8]) {
  float x[8], y[8];
  unpack8(a, x);
  unpack8(b, y);
  float u[8], v[8];
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
      u[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
      v[2 * i] = y[2 * i] * c[4 + i] - y[2 * i + 1] * s[4 + i];
      v[2 * i + 1] = y[2 * i + 1] * c[4 + i] + y[2 * i] * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = x[i] * c[i] - y[i] * s[i];
      v[i] = y[i] * c[i] + x[i] * s[i];
    }
  }
  a = pack8(u);
  b = pack8(v);
}

// Thread -> (token, head group, chunk), chunk fastest: neighbouring lanes read neighbouring
// vectors of a head, and the group's j-th head of neighbouring groups is neighbouring in memory.
// Heads are numbered through the tensors present: q, then k, then (append) v.
template <bool kInter, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  const uint32_t idx = blockIdx.x * static_cast<uint32_t>(kThreads) + threadIdx.x;
  if (idx >= a.units) return;
  const uint32_t item = idx / a.n_chunks;
  const int c = static_cast<int>(idx - item * a.n_chunks);
  const uint32_t tok32 = item / a.n_groups;
  const int g = static_cast<int>(item - tok32 * a.n_groups);
  const int64_t tok = a.tok0 + tok32;

  // the token's batch row and place, its position and (append) its cache slot
  int64_t b = 0, i = tok, pos;
  int64_t slot_k = -1;  // element offset of the token's row in the caches; < 0: not stored
  if (kAppend) {
    int n;
    if (a.cu) {
      // the sequence that owns row tok: the first whose end lies behind it
      int lo = 0, hi = a.B;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] <= tok) lo = mid + 1; else hi = mid;
      }
      if (lo >= a.B) return;  // rows behind the last sequence stay as they are
      b = lo;
      const int first = a.cu[lo];
      n = a.cu[lo + 1] - first;
      i = tok - first;
      if (i < 0) return;
    } else {
      b = a.B == 1 ? 0 : div_fl(tok, a.S);
      i = tok - b * a.S;
      n = static_cast<int>(a.S);
    }
    const int64_t j = static_cast<int64_t>(a.seq_len[b]) - n + i;
    pos = a.pos ? a.pos[tok] : a.pos0 + j;
    if (j >= 0) {
      const int64_t pg = div_fl(j, a.page_size);
      const int64_t page = pg < a.max_pages ? a.table[b * a.table_stride + pg] : -1;
      if (page >= 0 && page < a.n_pages)
        slot_k = page * a.page_stride + (j - pg * a.page_size) * a.slot_stride;
      else if (c == 0 && g == 0)
        atomicOr(a.err, kErrBadPage);
    }
    if (a.cu) {
      b = 0;  // packed rows: the inputs are addressed by row alone
      i = tok;
    }
  } else {
    b = a.B == 1 ? 0 : div_fl(tok, a.S);
    i = tok - b * a.S;
    pos = a.pos ? a.pos[tok] : a.pos0 + i;
  }

  // this chunk's two vectors of a head
  const int nr = a.rot >> 4;
  const bool turns = c < nr;
  int o0, o1;
  if (turns) {
    o0 = kInter ? 16 * c : 8 * c;
    o1 = kInter ? 16 * c + 8 : a.rot / 2 + 8 * c;
  } else {
    o0 = a.rot + 16 * (c - nr);
    o1 = o0 + 8;
  }
  const bool two = o1 < a.D;

  uint4 va[kHeads], vb[kHeads];
  __nv_bfloat16* out[kHeads];
  bool rot_head[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    int h = g + j * a.n_groups;
    out[j] = nullptr;
    rot_head[j] = turns;
    int t = 0;
    if (h >= a.heads[0]) {
      h -= a.heads[0];
      t = 1;
      if (h >= a.heads[1]) {
        h -= a.heads[1];
        t = 2;
        if (h >= a.heads[2]) continue;
      }
    }
    const __nv_bfloat16* src = a.src[t] + b * a.src_b[t] + i * a.src_s[t] + h * a.src_h[t];
    if (kAppend && t > 0) {
      if (slot_k < 0) continue;
      out[j] = a.dst[t] + slot_k + h * a.head_stride;
      if (t == 2) rot_head[j] = false;
    } else {
      out[j] = a.dst[t] + b * a.dst_b[t] + i * a.dst_s[t] + h * a.dst_h[t];
    }
    va[j] = *reinterpret_cast<const uint4*>(src + o0);
    if (two) vb[j] = *reinterpret_cast<const uint4*>(src + o1);
  }
  float cs[8], sn[8];
  if (turns) {
    const ulonglong2* ph = reinterpret_cast<const ulonglong2*>(a.phase) + 4 * c;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const ulonglong2 p = ph[q];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t t = static_cast<uint64_t>(pos) * (e ? p.y : p.x);
        const float half_turns = __ll2float_rn(static_cast<int64_t>(t)) * 0x1p-63f;
        float s_, c_;
        sincospif(half_turns, &s_, &c_);
        cs[2 * q + e] = c_ * a.mscale;
        sn[2 * q + e] = s_ * a.sin_scale;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    if (!out[j]) continue;
    if (rot_head[j]) rotate<kInter>(va[j], vb[j], cs, sn);
    *reinterpret_cast<uint4*>(out[j] + o0) = va[j];
    if (two) *reinterpret_cast<uint4*>(out[j] + o1) = vb[j];
  }
}

}  // namespace

cudaError_t launch_rope(RopeArgs a, bool interleaved, bool append, int64_t tokens,
                        cudaStream_t stream) {
  const int H = a.heads[0] + a.heads[1] + a.heads[2];
  const int nr = a.rot / 16;
  a.n_chunks = static_cast<uint32_t>(nr + (a.copy_tail ? (a.D - a.rot + 15) / 16 : 0));
  a.n_groups = static_cast<uint32_t>((H + kHeads - 1) / kHeads);
  const int64_t per_tok = static_cast<int64_t>(a.n_chunks) * a.n_groups;
  if (per_tok == 0 || tokens <= 0) return cudaSuccess;
  // unit indices fit 32 bits; a longer call goes in several launches
  const int64_t most = ((int64_t(1) << 31) - 1) / per_tok;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t n = tokens - t0 < most ? tokens - t0 : most;
    a.tok0 = t0;
    a.units = static_cast<uint32_t>(n * per_tok);
    const unsigned grid = static_cast<unsigned>((n * per_tok + kThreads - 1) / kThreads);
    launch_begin(append ? 12 : 11, stream);
    if (append) {
      if (interleaved) rope_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
      else rope_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
    } else {
      if (interleaved) rope_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
      else rope_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    launch_end(append ? 12 : 11, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace upipe
