// Device code that several kernels share: bf16 vectors as floats (the rotary, norm, embedding and log
// probability kernels), and where a token of a batch lies and goes (the first two).
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

}  // namespace upipe
