// C entries of the rotary positions, the paged key/value cache and the attention over it:
// argument checks (all before anything is enqueued), workspace plan and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "upipe.h"
#include "internal.h"

namespace upipe {
namespace {

int pfail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return status;
}

#define PAGED_CUDA(call)                                                         \
  do {                                                                           \
    cudaError_t e_ = (call);                                                     \
    if (e_ != cudaSuccess)                                                       \
      return pfail(UPIPE_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_));     \
  } while (0)

constexpr size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// The device pointers of one call, checked to be device memory of one device.
struct Placed {
  int dev = -1;
  int add(const void* p, const char* name, size_t align) {
    if (!p) return pfail(UPIPE_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
      return pfail(UPIPE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    pending[n] = p;
    names[n] = name;
    ++n;
    return UPIPE_OK;
  }
  // Looks the pointers up; after every check that needs no device.
  int resolve() {
    for (int i = 0; i < n; ++i) {
      cudaPointerAttributes at;
      if (cudaPointerGetAttributes(&at, pending[i]) != cudaSuccess) {
        cudaGetLastError();
        return pfail(UPIPE_ERR_INVALID_ARG, "%s must be device memory", names[i]);
      }
      if (at.type != cudaMemoryTypeDevice)
        return pfail(UPIPE_ERR_INVALID_ARG, "%s must be device memory", names[i]);
      if (dev < 0) dev = at.device;
      if (at.device != dev)
        return pfail(UPIPE_ERR_INVALID_ARG, "%s is on device %d, not %d", names[i], at.device, dev);
    }
    return UPIPE_OK;
  }
  const void* pending[20];
  const char* names[20];
  int n = 0;
};

// Whether rows of D elements at all combinations of three strides may overlap: unless each stride, in
// rising order, steps over all that the smaller ones span. (Layouts whose rows mesh without meeting
// are refused too; no permutation, slice or interleaving of dense tensors is one.)
bool may_overlap(const int64_t (&stride)[3], const int64_t (&extent)[3], int D) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] > stride[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1];
        order[j + 1] = t;
      }
  unsigned __int128 span = D;
  for (int i : order) {
    if (extent[i] <= 1) continue;
    if (static_cast<unsigned __int128>(stride[i]) < span) return true;
    span += static_cast<unsigned __int128>(stride[i]) * (extent[i] - 1);
  }
  return false;
}

// One strided [B, S, heads, D] tensor. Written ones must not overlap themselves.
int check_heads(const upipe_heads* t, const char* name, int64_t B, int64_t S, int D, bool written,
                Placed* p) {
  if (t->heads < 1) return pfail(UPIPE_ERR_INVALID_ARG, "%s has %d heads", name, t->heads);
  const int64_t st[3] = {t->stride_b, t->stride_s, t->stride_h};
  const int64_t ext[3] = {B, S, t->heads};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] <= 1) continue;
    if (st[i] < 0 || st[i] % 8)
      return pfail(UPIPE_ERR_INVALID_ARG,
                   "%s: strides must be multiples of 8 elements and not negative", name);
    if (written && st[i] < D)
      return pfail(UPIPE_ERR_INVALID_ARG, "%s: a written tensor's strides must be at least D", name);
  }
  if (written && may_overlap(st, ext, D))
    return pfail(UPIPE_ERR_INVALID_ARG, "%s: a written tensor must not overlap itself", name);
  return p->add(t->data, name, 16);
}

void set_view(RopeArgs* a, int i, const upipe_heads* src, const upipe_heads* dst) {
  a->heads[i] = src->heads;
  a->src[i] = static_cast<const __nv_bfloat16*>(src->data);
  a->src_b[i] = src->stride_b;
  a->src_s[i] = src->stride_s;
  a->src_h[i] = src->stride_h;
  if (!dst) return;
  a->dst[i] = static_cast<__nv_bfloat16*>(dst->data);
  a->dst_b[i] = dst->stride_b;
  a->dst_s[i] = dst->stride_s;
  a->dst_h[i] = dst->stride_h;
}

bool same_place(const upipe_heads* x, const upipe_heads* y) {
  return x->data == y->data && x->stride_b == y->stride_b && x->stride_s == y->stride_s &&
         x->stride_h == y->stride_h;
}

bool present(const upipe_heads* t) { return t && t->heads != 0; }

int check_rot(int D, int rot) {
  if (D < 8 || D > 1024 || D % 8)
    return pfail(UPIPE_ERR_UNSUPPORTED, "D=%d (supported: multiples of 8 up to 1024)", D);
  if (rot < 16 || rot > D || rot % 16)
    return pfail(UPIPE_ERR_UNSUPPORTED, "rot_dim=%d (supported: multiples of 16 up to D)", rot);
  return UPIPE_OK;
}

int rope(const char* where, const upipe_heads* q, const upipe_heads* k, const upipe_heads* q_out,
         const upipe_heads* k_out, const int64_t* pos, int64_t pos0, const uint64_t* phase,
         double mscale, int B, int64_t S, int D, int rot, int interleaved, bool back,
         void* stream) {
  const NvtxRange range(where);
  set_last_error("");
  if (B < 0 || S < 0) return pfail(UPIPE_ERR_INVALID_ARG, "B=%d S=%lld", B, (long long)S);
  if (B > 0 && S > (int64_t(1) << 40) / B)
    return pfail(UPIPE_ERR_UNSUPPORTED, "more than 2^40 tokens");
  int st = check_rot(D, rot);
  if (st != UPIPE_OK) return st;
  if (interleaved != 0 && interleaved != 1)
    return pfail(UPIPE_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!std::isfinite(mscale)) return pfail(UPIPE_ERR_INVALID_ARG, "mscale must be finite");
  const bool has_q = present(q), has_k = present(k);
  if (!has_q && !has_k) return pfail(UPIPE_ERR_INVALID_ARG, "neither q nor k");
  if ((has_q && !present(q_out)) || (has_k && !present(k_out)))
    return pfail(UPIPE_ERR_INVALID_ARG, "an input without its output");
  if (B == 0 || S == 0) return UPIPE_OK;
  if ((has_q ? static_cast<int64_t>(q->heads) : 0) + (has_k ? k->heads : 0) > 65536)
    return pfail(UPIPE_ERR_UNSUPPORTED, "more than 65536 heads");
  Placed p;
  RopeArgs a{};
  bool in_place = true;
  const upipe_heads* in[2] = {q, k};
  const upipe_heads* out[2] = {q_out, k_out};
  const char* names[4] = {"q", "k", "q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    if (!present(in[i])) continue;
    if (in[i]->heads != out[i]->heads)
      return pfail(UPIPE_ERR_INVALID_ARG, "%s and %s differ in heads", names[i], names[2 + i]);
    st = check_heads(in[i], names[i], B, S, D, false, &p);
    if (st == UPIPE_OK) st = check_heads(out[i], names[2 + i], B, S, D, true, &p);
    if (st != UPIPE_OK) return st;
    set_view(&a, i, in[i], out[i]);
    in_place = in_place && same_place(in[i], out[i]);
  }
  if (has_q && has_k && q_out->data == k_out->data)
    return pfail(UPIPE_ERR_INVALID_ARG, "q_out and k_out are one tensor");
  st = p.add(phase, "phase", 16);
  if (st == UPIPE_OK && pos) st = p.add(pos, "pos", 8);
  if (st == UPIPE_OK) st = p.resolve();
  if (st != UPIPE_OK) return st;
  a.B = B;
  a.S = S;
  a.D = D;
  a.rot = rot;
  a.copy_tail = rot < D && !in_place;
  a.pos = pos;
  a.pos0 = pos0;
  a.phase = phase;
  a.mscale = static_cast<float>(mscale);
  a.sin_scale = back ? -a.mscale : a.mscale;
  const DeviceGuard dguard;
  PAGED_CUDA(cudaSetDevice(p.dev));
  PAGED_CUDA(launch_rope(a, interleaved != 0, false, static_cast<int64_t>(B) * S,
                         static_cast<cudaStream_t>(stream)));
  return UPIPE_OK;
}

int check_pages(const upipe_pages* c, Placed* p) {
  if (!c) return pfail(UPIPE_ERR_INVALID_ARG, "cache is NULL");
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff || c->page_size < 1 || c->heads < 1)
    return pfail(UPIPE_ERR_INVALID_ARG, "cache: n_pages=%lld page_size=%d heads=%d",
                 (long long)c->n_pages, c->page_size, c->heads);
  const int64_t st[3] = {c->stride_page, c->stride_slot, c->stride_head};
  for (int i = 0; i < 3; ++i)
    if (st[i] < c->D || st[i] % 8 || st[i] >= (int64_t(1) << 39))
      return pfail(UPIPE_ERR_INVALID_ARG,
                   "cache: strides must be multiples of 8 elements, at least D and below 2^39");
  int r = p->add(c->k, "cache.k", 16);
  if (r == UPIPE_OK) r = p->add(c->v, "cache.v", 16);
  return r;
}

int gcd(int x, int y) {
  while (y) {
    const int t = x % y;
    x = y;
    y = t;
  }
  return x;
}

// Byte offsets of an attention call's workspace, each 256-byte aligned.
struct PagedPlan {
  size_t px_o, px_ml, slot_o, slot_ml, desc, total;
};

// Shape checks and plan of an attention call (no device access).
int attn_plan(int B, int64_t rows, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_q,
              int64_t max_len, PagedArgs* a, PagedPlan* p) {
  if (B < 1 || rows < 1 || Hq < 1 || Hkv < 1 || D < 1 || prefix_len < 0 || max_q < 1 ||
      max_len < 1)
    return pfail(UPIPE_ERR_INVALID_ARG,
                 "B=%d rows=%lld Hq=%d Hkv=%d D=%d prefix_len=%lld max_q=%lld max_len=%lld", B,
                 (long long)rows, Hq, Hkv, D, (long long)prefix_len, (long long)max_q,
                 (long long)max_len);
  if (Hq % Hkv) return pfail(UPIPE_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (D != 64 && D != 128)
    return pfail(UPIPE_ERR_UNSUPPORTED, "D=%d (supported: 64, 128)", D);
  if (prefix_len > (int64_t(1) << 30) || rows > (int64_t(1) << 24) || Hq > 4096 || B > (1 << 20))
    return pfail(UPIPE_ERR_UNSUPPORTED,
                 "prefix_len=%lld rows=%lld Hq=%d B=%d (at most 2^30, 2^24, 4096, 2^20)",
                 (long long)prefix_len, (long long)rows, Hq, B);
  a->B = B;
  a->rows = rows;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->G = Hq / Hkv;
  a->D = D;
  a->prefix = prefix_len;
  plan_paged(a, max_q < rows ? max_q : rows, max_len);
  if (a->n_slots * a->mt > 0x7fffffff ||
      static_cast<int64_t>(a->Hkv) * a->tiles_p * a->splits_x > 0x7fffffff)
    return pfail(UPIPE_ERR_UNSUPPORTED, "B=%d rows=%lld Hq=%d: too many row tiles", B,
                 (long long)rows, Hq);
  const size_t px = static_cast<size_t>(a->splits_p) * rows * Hq;
  const size_t sl = static_cast<size_t>(a->n_slots) * a->mt;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += al256(bytes);
    return at;
  };
  p->px_o = take(px * D * 4);
  p->px_ml = take(px * 16);
  p->slot_o = take(sl * D * 4);
  p->slot_ml = take(sl * 16);
  p->desc = take(2 * static_cast<size_t>(rows) * Hq * 8);
  p->total = off;
  return UPIPE_OK;
}

// f / (2 pi) modulo 1 in units of 2^-64, rounded to nearest. A double holds 11 bits too few for it, so
// the quotient is kept as a sum q + e of two: e = (f - q 2 pi) / 2 pi, with 2 pi as a sum of two
// doubles and the remainder by fused multiply-adds (the first of which is exact). q + e is then
// within 2^-103 of itself: less than 2^-2 units for every |f| below 2^40.
uint64_t phase_of(double f) {
  const double p = 6.283185307179586, p_low = 2.4492935982947064e-16;
  const double x = std::fabs(f);
  double q = x / p;
  double e = std::fma(-q, p_low, std::fma(-q, p, x)) / p;
  // whole turns do not count: both steps are exact
  q -= std::floor(q);
  e -= std::rint(e);
  const double units = std::ldexp(q, 64), whole = std::floor(units);
  double rest = std::rint((units - whole) + std::ldexp(e, 64));
  if (rest >= 0x1p63) rest -= 0x1p64;
  const uint64_t w = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(rest));
  return f < 0.0 ? 0 - w : w;
}

}  // namespace
}  // namespace upipe

using namespace upipe;

extern "C" {

int upipe_rope_frequencies(double* inv_freq, double* mscale, int rot_dim, double theta,
                           int scaling, double factor, double trained_len, double turns_fast,
                           double turns_slow) {
  set_last_error("");
  if (!inv_freq || !mscale) return pfail(UPIPE_ERR_INVALID_ARG, "inv_freq or mscale is NULL");
  if (rot_dim < 2 || rot_dim % 2) return pfail(UPIPE_ERR_INVALID_ARG, "rot_dim=%d", rot_dim);
  if (!(theta > 1.0) || !std::isfinite(theta))
    return pfail(UPIPE_ERR_INVALID_ARG, "theta must be above 1");
  if (scaling < UPIPE_ROPE_PLAIN || scaling > UPIPE_ROPE_BY_PARTS)
    return pfail(UPIPE_ERR_INVALID_ARG, "scaling=%d", scaling);
  if (scaling != UPIPE_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return pfail(UPIPE_ERR_INVALID_ARG, "factor must be at least 1");
  if (scaling == UPIPE_ROPE_NTK && rot_dim < 4)
    return pfail(UPIPE_ERR_INVALID_ARG, "rot_dim=%d is too small for this scaling", rot_dim);
  if (scaling == UPIPE_ROPE_BY_PARTS && (!(trained_len > 0.0) || !(turns_fast > turns_slow)))
    return pfail(UPIPE_ERR_INVALID_ARG, "trained_len must be positive and turns_fast above turns_slow");
  const double pi = 3.14159265358979323846;
  if (scaling == UPIPE_ROPE_NTK) theta *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == UPIPE_ROPE_LINEAR) f /= factor;
    if (scaling == UPIPE_ROPE_BY_PARTS) {
      double g = (trained_len * f / (2.0 * pi) - turns_slow) / (turns_fast - turns_slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f *= g + (1.0 - g) / factor;
    }
    inv_freq[i] = f;
  }
  *mscale = scaling == UPIPE_ROPE_BY_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return UPIPE_OK;
}

int upipe_rope_phases(const double* inv_freq, uint64_t* phase, int n) {
  set_last_error("");
  if (!inv_freq || !phase) return pfail(UPIPE_ERR_INVALID_ARG, "inv_freq or phase is NULL");
  if (n < 1) return pfail(UPIPE_ERR_INVALID_ARG, "n=%d", n);
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i]))
      return pfail(UPIPE_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
    phase[i] = phase_of(inv_freq[i]);
  }
  return UPIPE_OK;
}

int upipe_rope_fwd(const upipe_heads* q, const upipe_heads* k, const upipe_heads* q_out,
                   const upipe_heads* k_out, const int64_t* pos, int64_t pos0,
                   const uint64_t* phase, double mscale, int B, int64_t S, int D, int rot_dim,
                   int interleaved, void* stream) {
  return rope("upipe_rope_fwd", q, k, q_out, k_out, pos, pos0, phase, mscale, B, S, D, rot_dim,
              interleaved, false, stream);
}

int upipe_rope_bwd(const upipe_heads* dq_out, const upipe_heads* dk_out, const upipe_heads* dq,
                   const upipe_heads* dk, const int64_t* pos, int64_t pos0, const uint64_t* phase,
                   double mscale, int B, int64_t S, int D, int rot_dim, int interleaved,
                   void* stream) {
  return rope("upipe_rope_bwd", dq_out, dk_out, dq, dk, pos, pos0, phase, mscale, B, S, D, rot_dim,
              interleaved, true, stream);
}

int upipe_kv_append(const upipe_heads* q, const upipe_heads* q_out, const upipe_heads* k,
                    const upipe_heads* v, const upipe_pages* cache, const int32_t* page_table,
                    int64_t table_stride, int64_t max_pages, const int32_t* seq_len,
                    const int32_t* cu_rows, const int64_t* pos, int64_t pos0,
                    const uint64_t* phase, double mscale, int B, int64_t S, int rot_dim,
                    int interleaved, void* stream) {
  const NvtxRange range("upipe_kv_append");
  set_last_error("");
  if (B < 0 || S < 0) return pfail(UPIPE_ERR_INVALID_ARG, "B=%d S=%lld", B, (long long)S);
  if (S > 0x7fffffff || (B > 0 && S > (int64_t(1) << 40) / B))
    return pfail(UPIPE_ERR_UNSUPPORTED, "more than 2^31 rows a sequence or 2^40 rows");
  if (!present(k) || !present(v)) return pfail(UPIPE_ERR_INVALID_ARG, "k or v is missing");
  if (interleaved != 0 && interleaved != 1)
    return pfail(UPIPE_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  Placed p;
  int st = check_pages(cache, &p);
  if (st != UPIPE_OK) return st;
  const int D = cache->D;
  if (phase) {
    st = check_rot(D, rot_dim);
    if (st != UPIPE_OK) return st;
    if (!std::isfinite(mscale)) return pfail(UPIPE_ERR_INVALID_ARG, "mscale must be finite");
  } else if (D < 8 || D > 1024 || D % 8) {
    return pfail(UPIPE_ERR_UNSUPPORTED, "D=%d (supported: multiples of 8 up to 1024)", D);
  }
  if (k->heads != cache->heads || v->heads != cache->heads)
    return pfail(UPIPE_ERR_INVALID_ARG, "k and v have %d and %d heads, the cache %d", k->heads,
                 v->heads, cache->heads);
  const bool has_q = present(q);
  if (has_q && (!present(q_out) || q_out->heads != q->heads))
    return pfail(UPIPE_ERR_INVALID_ARG, "q_out is missing or differs from q in heads");
  if (2 * static_cast<int64_t>(k->heads) + (has_q ? q->heads : 0) > 65536)
    return pfail(UPIPE_ERR_UNSUPPORTED, "more than 65536 heads");
  if (max_pages < 1 || (B > 1 && table_stride < max_pages))
    return pfail(UPIPE_ERR_INVALID_ARG, "max_pages=%lld table_stride=%lld", (long long)max_pages,
                 (long long)table_stride);
  if (may_overlap({cache->stride_page, cache->stride_slot, cache->stride_head},
                  {cache->n_pages, cache->page_size, cache->heads}, D))
    return pfail(UPIPE_ERR_INVALID_ARG, "cache: pages, slots or heads overlap");
  if (B == 0 || S == 0) return UPIPE_OK;
  const int64_t vb = cu_rows ? 1 : B;
  RopeArgs a{};
  if (has_q) {
    st = check_heads(q, "q", vb, S, D, false, &p);
    if (st == UPIPE_OK) st = check_heads(q_out, "q_out", vb, S, D, true, &p);
    if (st != UPIPE_OK) return st;
    set_view(&a, 0, q, q_out);
  }
  st = check_heads(k, "k", vb, S, D, false, &p);
  if (st == UPIPE_OK) st = check_heads(v, "v", vb, S, D, false, &p);
  if (st == UPIPE_OK) st = p.add(page_table, "page_table", 4);
  if (st == UPIPE_OK) st = p.add(seq_len, "seq_len", 4);
  if (st == UPIPE_OK && cu_rows) st = p.add(cu_rows, "cu_rows", 4);
  if (st == UPIPE_OK && pos) st = p.add(pos, "pos", 8);
  if (st == UPIPE_OK && phase) st = p.add(phase, "phase", 16);
  if (st == UPIPE_OK) st = p.resolve();
  if (st != UPIPE_OK) return st;
  set_view(&a, 1, k, nullptr);
  set_view(&a, 2, v, nullptr);
  a.dst[1] = static_cast<__nv_bfloat16*>(cache->k);
  a.dst[2] = static_cast<__nv_bfloat16*>(cache->v);
  a.B = B;
  a.S = S;
  a.D = D;
  a.rot = phase ? rot_dim : 0;
  a.copy_tail = a.rot < D;
  a.pos = pos;
  a.pos0 = pos0;
  a.phase = phase;
  a.mscale = a.sin_scale = static_cast<float>(mscale);
  a.table = page_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.page_stride = cache->stride_page;
  a.slot_stride = cache->stride_slot;
  a.head_stride = cache->stride_head;
  a.seq_len = seq_len;
  a.cu = cu_rows;
  const DeviceGuard dguard;
  PAGED_CUDA(cudaSetDevice(p.dev));
  st = device_status_word(p.dev, &a.err);
  if (st != UPIPE_OK) return st;
  PAGED_CUDA(launch_rope(a, interleaved != 0, true, cu_rows ? S : static_cast<int64_t>(B) * S,
                         static_cast<cudaStream_t>(stream)));
  return UPIPE_OK;
}

size_t upipe_attn_paged_workspace_bytes(int B, int64_t rows, int Hq, int Hkv, int D,
                                        int64_t prefix_len, int64_t max_q, int64_t max_len) {
  PagedArgs a{};
  PagedPlan p{};
  return attn_plan(B, rows, Hq, Hkv, D, prefix_len, max_q, max_len, &a, &p) == UPIPE_OK ? p.total : 0;
}

int upipe_attn_paged_fwd(const upipe_heads* q, const upipe_heads* o, float* lse,
                         const upipe_pages* cache, const int32_t* page_table,
                         int64_t table_stride, int64_t max_pages, const int32_t* seq_len,
                         const int32_t* cu_rows, const int32_t* prefix_table, int64_t prefix_len,
                         int B, int64_t S, int64_t max_q, int64_t max_len, void* workspace,
                         size_t workspace_bytes, void* stream_) {
  const NvtxRange range("upipe_attn_paged_fwd");
  set_last_error("");
  if (B < 0 || S < 0) return pfail(UPIPE_ERR_INVALID_ARG, "B=%d S=%lld", B, (long long)S);
  if (!present(q) || !present(o)) return pfail(UPIPE_ERR_INVALID_ARG, "q or o is missing");
  if (q->heads != o->heads) return pfail(UPIPE_ERR_INVALID_ARG, "q and o differ in heads");
  Placed p;
  int st = check_pages(cache, &p);
  if (st != UPIPE_OK) return st;
  if (cache->page_size % 16)
    return pfail(UPIPE_ERR_UNSUPPORTED, "page_size=%d (supported: multiples of 16)",
                 cache->page_size);
  if (max_pages < 1 || (B > 1 && table_stride < max_pages))
    return pfail(UPIPE_ERR_INVALID_ARG, "max_pages=%lld table_stride=%lld", (long long)max_pages,
                 (long long)table_stride);
  if (B == 0 || S == 0) return UPIPE_OK;
  if (S > (int64_t(1) << 24))
    return pfail(UPIPE_ERR_UNSUPPORTED, "S=%lld (at most 2^24)", (long long)S);
  PagedArgs a{};
  const int64_t rows = cu_rows ? S : static_cast<int64_t>(B) * S;
  if (!cu_rows) max_q = S;
  PagedPlan plan{};
  st = attn_plan(B, rows, q->heads, cache->heads, cache->D, prefix_len, max_q, max_len, &a,
                 &plan);
  if (st != UPIPE_OK) return st;
  const int D = cache->D;
  const int64_t vb = cu_rows ? 1 : B;
  st = check_heads(q, "q", vb, S, D, false, &p);
  if (st == UPIPE_OK) st = check_heads(o, "o", vb, S, D, true, &p);
  if (st == UPIPE_OK && lse) st = p.add(lse, "lse", 4);
  if (st == UPIPE_OK) st = p.add(page_table, "page_table", 4);
  if (st == UPIPE_OK) st = p.add(seq_len, "seq_len", 4);
  if (st == UPIPE_OK && cu_rows) st = p.add(cu_rows, "cu_rows", 4);
  if (st == UPIPE_OK && prefix_len) st = p.add(prefix_table, "prefix_table", 4);
  if (st == UPIPE_OK) st = p.add(workspace, "workspace", 256);
  if (st != UPIPE_OK) return st;
  a.cap = max_pages > kMaxOwnKeys / cache->page_size
              ? kMaxOwnKeys
              : static_cast<int>(max_pages * cache->page_size);
  // the kernels count in 32 bits: a segment's tiles (rounded up) and kSegmentCost more
  const double tiles =
      static_cast<double>(a.segs) * (a.cap / a.ks + 1.0 + kSegmentCost) +
      static_cast<double>(a.segs_p) * (static_cast<double>(prefix_len) / a.ks + 1.0 + kSegmentCost);
  if (tiles >= 4294967296.0)
    return pfail(UPIPE_ERR_UNSUPPORTED,
                 "%lld row tiles of up to %d keys: more than 2^32 tiles (use narrower page tables)",
                 (long long)a.segs, a.cap);
  if (workspace_bytes < plan.total)
    return pfail(UPIPE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes,
                 plan.total);
  st = p.resolve();
  if (st != UPIPE_OK) return st;
  a.q = static_cast<const __nv_bfloat16*>(q->data);
  a.q_b = q->stride_b;
  a.q_s = q->stride_s;
  a.q_h = q->stride_h;
  a.o = static_cast<__nv_bfloat16*>(o->data);
  a.o_b = o->stride_b;
  a.o_s = o->stride_s;
  a.o_h = o->stride_h;
  a.kc = static_cast<const __nv_bfloat16*>(cache->k);
  a.vc = static_cast<const __nv_bfloat16*>(cache->v);
  a.page_stride = cache->stride_page;
  a.slot_stride = cache->stride_slot;
  a.head_stride = cache->stride_head;
  a.lse = lse;
  a.T = S;
  a.cu = cu_rows;
  a.table = page_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.n_pages = cache->n_pages;
  a.seq_len = seq_len;
  a.ptable = prefix_table;
  a.page_size = cache->page_size;
  a.scale_log2 = 1.0f / std::sqrt(static_cast<float>(D)) * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + plan.px_o);
  a.part_ml = reinterpret_cast<float4*>(ws + plan.px_ml);
  a.slot_o = reinterpret_cast<float*>(ws + plan.slot_o);
  a.slot_ml = reinterpret_cast<float4*>(ws + plan.slot_ml);
  a.desc = reinterpret_cast<int2*>(ws + plan.desc);
  const DeviceGuard dguard;
  PAGED_CUDA(cudaSetDevice(p.dev));
  st = device_status_word(p.dev, &a.err);
  if (st != UPIPE_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  auto maps = [&](CUtensorMap* km, CUtensorMap* vm, int box_rows) -> cudaError_t {
    cudaError_t e = make_tmap_pages(km, cache->k, D, cache->page_size, cache->heads,
                                    cache->n_pages, cache->stride_slot, cache->stride_head,
                                    cache->stride_page, box_rows);
    if (e != cudaSuccess) return e;
    return make_tmap_pages(vm, cache->v, D, cache->page_size, cache->heads, cache->n_pages,
                           cache->stride_slot, cache->stride_head, cache->stride_page, box_rows);
  };
  CUtensorMap km, vm;
  if (a.splits_x) {
    a.box_rows = gcd(cache->page_size, 128);
    PAGED_CUDA(maps(&km, &vm, a.box_rows));
    PAGED_CUDA(launch_attn_prefix(a, km, vm, stream));
  }
  if (a.mt == 64) {
    a.box_rows = gcd(cache->page_size, a.ks);
    PAGED_CUDA(maps(&km, &vm, a.box_rows));
  }
  PAGED_CUDA(launch_attn_paged(a, &km, &vm, stream));
  PAGED_CUDA(launch_paged_merge(a, stream));
  return UPIPE_OK;
}

}  // extern "C"
