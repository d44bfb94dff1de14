// Device code that the rotary kernels share: the bf16 vectors, the rotation of eight pairs, the
// angles of a position, and where a token of a batch lies and goes.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace upipe {

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// Two vectors x, y of one head that hold eight pairs: (x_i, y_i) in the half layout,
// consecutive elements of x and then of y in the interleaved one.
template <bool kInter>
__device__ __forceinline__ void rotate_pairs(float (&x)[8], float (&y)[8], const float (&c)[8],
                                             const float (&s)[8]) {
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
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = u[i];
    y[i] = v[i];
  }
}

// Factors of chunk c's eight pairs at position pos (see rope.cu on the angles).
__device__ __forceinline__ void chunk_angles(const uint64_t* phase, int c, int64_t pos,
                                             float mscale, float sin_scale, float (&cs)[8],
                                             float (&sn)[8]) {
  const ulonglong2* ph = reinterpret_cast<const ulonglong2*>(phase) + 4 * c;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const ulonglong2 p = ph[q];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t t = static_cast<uint64_t>(pos) * (e ? p.y : p.x);
      const float half_turns = __ll2float_rn(static_cast<int64_t>(t)) * 0x1p-63f;
      float s_, c_;
      sincospif(half_turns, &s_, &c_);
      cs[2 * q + e] = c_ * mscale;
      sn[2 * q + e] = s_ * sin_scale;
    }
  }
}

// Batch row and place of a token (packed rows of an append: row 0, the token itself), its position
// and, for an append, the element offset of its slot in the caches (< 0: not stored).
struct TokenPlace {
  int64_t b, i, pos, slot;
};

// False: a row that no sequence owns. report: this thread reports a page that does not exist.
template <bool kAppend>
__device__ __forceinline__ bool place_token(const RopeArgs& a, int64_t tok, bool report,
                                            TokenPlace* p) {
  int64_t b = 0, i = tok;
  p->slot = -1;
  if (kAppend) {
    int n;
    if (a.cu) {
      // the sequence that owns row tok: the first whose end lies behind it
      int lo = 0, hi = a.B;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] <= tok) lo = mid + 1; else hi = mid;
      }
      if (lo >= a.B) return false;  // rows behind the last sequence stay as they are
      b = lo;
      const int first = a.cu[lo];
      n = a.cu[lo + 1] - first;
      i = tok - first;
      if (i < 0) return false;
    } else {
      b = a.B == 1 ? 0 : div_fl(tok, a.S);
      i = tok - b * a.S;
      n = static_cast<int>(a.S);
    }
    const int64_t j = static_cast<int64_t>(a.seq_len[b]) - n + i;
    p->pos = a.pos ? a.pos[tok] : a.pos0 + j;
    if (j >= 0) {
      const int64_t pg = div_fl(j, a.page_size);
      const int64_t page = pg < a.max_pages ? a.table[b * a.table_stride + pg] : -1;
      if (page >= 0 && page < a.n_pages)
        p->slot = page * a.page_stride + (j - pg * a.page_size) * a.slot_stride;
      else if (report)
        atomicOr(a.err, kErrBadPage);
    }
    if (a.cu) {
      b = 0;  // packed rows: the inputs are addressed by row alone
      i = tok;
    }
  } else {
    b = a.B == 1 ? 0 : div_fl(tok, a.S);
    i = tok - b * a.S;
    p->pos = a.pos ? a.pos[tok] : a.pos0 + i;
  }
  p->b = b;
  p->i = i;
  return true;
}

// The two vectors of a head that chunk c holds: a turning chunk's pairs, or (behind the rotated
// part) sixteen features in a row.
__device__ __forceinline__ bool chunk_features(int c, int rot, bool inter, int* o0, int* o1) {
  const int nr = rot >> 4;
  if (c < nr) {
    *o0 = inter ? 16 * c : 8 * c;
    *o1 = inter ? 16 * c + 8 : rot / 2 + 8 * c;
    return true;
  }
  *o0 = rot + 16 * (c - nr);
  *o1 = *o0 + 8;
  return false;
}

}  // namespace upipe
