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
// Bound: HBM. A thread owns the 16 features of a chunk (two 16-byte vectors, eight pairs) of a few
// heads of one token, and the 2, 4, 8, 16 or 32 lanes that share a head add up its sums by shuffles.
// Heads of one tensor form a thread's group, so the weights of its chunk are read once.
#include "internal.h"
#include "rope.cuh"

namespace upipe {
namespace {

constexpr int kFwdThreads = 64;
constexpr int kFwdHeads = 4;  // heads of one token per thread
constexpr int kBwdThreads = 256;
constexpr int kBwdHeads = 2;

// A chunk's effective weights: offset + w, or ones.
__device__ __forceinline__ void load_weights(const NormArgs& a, int t, int o, float (&w)[8]) {
  if (!a.w[t]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    return;
  }
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

__device__ __forceinline__ float dot8(const float (&x)[8], const float (&y)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  return s;
}

// Sum over the lanes that share a head.
__device__ __forceinline__ float head_sum(float s, int lanes) {
  for (int m = lanes >> 1; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}

// (ss / D + eps)^(-1/2) of a head whose squares sum to ss; heads whose squares leave fp32's range
// (elements of 2^59 and more) are summed again, scaled down by 2^96. All lanes of a warp call.
__device__ __forceinline__ float inverse_rms(const NormArgs& a, float ss, const float (&x)[8],
                                             const float (&y)[8]) {
  float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
  const bool out = !(ss <= 0x1p127f);
  if (__any_sync(0xffffffffu, out)) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x[i] * 0x1p-96f, v = y[i] * 0x1p-96f;
      s += u * u + v * v;
    }
    s = head_sum(s, a.lanes);
    if (out) r = 0x1p-96f * rsqrtf(s * a.inv_d);
  }
  return r;
}

// Thread -> (token, head group, lane of a head), lane fastest; groups number q's, k's, v's heads.
template <bool kInter, bool kAppend>
__global__ void __launch_bounds__(kFwdThreads) norm_rope_kernel(const NormArgs a) {
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
  const bool turns = chunk_features(c, ra.rot, kInter, &o0, &o1);
  const bool in0 = o0 < ra.D, two = o1 < ra.D;

  uint4 va[kFwdHeads], vb[kFwdHeads];
  __nv_bfloat16* out[kFwdHeads];
#pragma unroll
  for (int j = 0; j < kFwdHeads; ++j) {
    const int h = g + j * a.groups[t];
    out[j] = nullptr;
    va[j] = vb[j] = make_uint4(0, 0, 0, 0);
    if (!live || !in0 || h >= ra.heads[t]) continue;
    if (kAppend && t > 0) {
      if (at.slot < 0) continue;
      out[j] = ra.dst[t] + at.slot + h * ra.head_stride;
    } else {
      out[j] = ra.dst[t] + at.b * ra.dst_b[t] + at.i * ra.dst_s[t] + h * ra.dst_h[t];
    }
    const __nv_bfloat16* src = ra.src[t] + at.b * ra.src_b[t] + at.i * ra.src_s[t] + h * ra.src_h[t];
    va[j] = *reinterpret_cast<const uint4*>(src + o0);
    if (two) vb[j] = *reinterpret_cast<const uint4*>(src + o1);
  }
  float cs[8], sn[8], wa[8], wb[8];
  const bool normed = t < 2;
  if (live && in0 && normed) {
    if (turns) chunk_angles(ra.phase, c, at.pos, ra.mscale, ra.sin_scale, cs, sn);
    load_weights(a, t, o0, wa);
    if (two) load_weights(a, t, o1, wb);
  }
#pragma unroll
  for (int j = 0; j < kFwdHeads; ++j) {
    float x[8], y[8];
    unpack_bf16x8(va[j], x);
    unpack_bf16x8(vb[j], y);
    const float ss = head_sum(dot8(x, x) + dot8(y, y), a.lanes);
    const float r = inverse_rms(a, normed ? ss : 0.f, x, y);
    if (!out[j]) continue;
    if (normed) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = x[i] * r * wa[i];
        y[i] = y[i] * r * wb[i];
      }
      if (turns) rotate_pairs<kInter>(x, y, cs, sn);
      va[j] = pack_bf16x8(x);
      vb[j] = pack_bf16x8(y);
    }
    *reinterpret_cast<uint4*>(out[j] + o0) = va[j];
    if (two) *reinterpret_cast<uint4*>(out[j] + o1) = vb[j];
  }
}

// A set of `lanes` lanes keeps one head group and walks the tokens, so that its 16 sums of dw and its
// weights stay in registers; a block adds its sets' sums in order and leaves 2 D partial sums.
template <bool kInter>
__global__ void __launch_bounds__(kBwdThreads, 2) norm_rope_bwd_kernel(const NormArgs a) {
  const RopeArgs& ra = a.r;
  __shared__ float part[kBwdThreads * 16];
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
  const bool turns = chunk_features(c, ra.rot, kInter, &o0, &o1);
  const bool in0 = o0 < ra.D, two = o1 < ra.D;
  float wa[8], wb[8], da[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wa[i] = wb[i] = da[i] = db[i] = 0.f;
  if (in0) load_weights(a, t, o0, wa);
  if (two) load_weights(a, t, o1, wb);

  // every lane of a warp takes the same number of steps: the shuffles want them all
  const int64_t steps = (a.tokens + walkers - 1) / walkers;
  for (int64_t n = 0; n < steps; ++n) {
    const int64_t tok = n * walkers + walker;
    const bool live = walker < walkers && tok < a.tokens && in0;
    TokenPlace at{};
    if (live) place_token<false>(ra, tok, false, &at);
    uint4 xa[kBwdHeads], xb[kBwdHeads], ga[kBwdHeads], gb[kBwdHeads];
#pragma unroll
    for (int j = 0; j < kBwdHeads; ++j) {
      const int h = g + j * a.groups[t];
      xa[j] = xb[j] = ga[j] = gb[j] = make_uint4(0, 0, 0, 0);
      if (!live || h >= ra.heads[t]) continue;
      const __nv_bfloat16* x = a.x[t] + at.b * a.x_b[t] + at.i * a.x_s[t] + h * a.x_h[t];
      const __nv_bfloat16* dy = ra.src[t] + at.b * ra.src_b[t] + at.i * ra.src_s[t] + h * ra.src_h[t];
      xa[j] = *reinterpret_cast<const uint4*>(x + o0);
      ga[j] = *reinterpret_cast<const uint4*>(dy + o0);
      if (two) {
        xb[j] = *reinterpret_cast<const uint4*>(x + o1);
        gb[j] = *reinterpret_cast<const uint4*>(dy + o1);
      }
    }
    float cs[8], sn[8];
    if (live && turns) chunk_angles(ra.phase, c, at.pos, ra.mscale, ra.sin_scale, cs, sn);
#pragma unroll
    for (int j = 0; j < kBwdHeads; ++j) {
      const int h = g + j * a.groups[t];
      float x[8], y[8], u[8], v[8];
      unpack_bf16x8(xa[j], x);
      unpack_bf16x8(xb[j], y);
      unpack_bf16x8(ga[j], u);
      unpack_bf16x8(gb[j], v);
      if (live && turns) rotate_pairs<kInter>(u, v, cs, sn);
      const float ss = head_sum(dot8(x, x) + dot8(y, y), a.lanes);
      const float r = inverse_rms(a, ss, x, y);
      float tx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= r;
        y[i] *= r;
        da[i] = fmaf(u[i], x[i], da[i]);
        db[i] = fmaf(v[i], y[i], db[i]);
        u[i] *= wa[i];
        v[i] *= wb[i];
        tx = fmaf(u[i], x[i], fmaf(v[i], y[i], tx));
      }
      tx = head_sum(tx, a.lanes) * a.inv_d;
      if (!live || h >= ra.heads[t]) continue;
      __nv_bfloat16* dx = ra.dst[t] + at.b * ra.dst_b[t] + at.i * ra.dst_s[t] + h * ra.dst_h[t];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = r * fmaf(-x[i], tx, u[i]);
        v[i] = r * fmaf(-y[i], tx, v[i]);
      }
      *reinterpret_cast<uint4*>(dx + o0) = pack_bf16x8(u);
      if (two) *reinterpret_cast<uint4*>(dx + o1) = pack_bf16x8(v);
    }
  }

  if (!a.part) return;
  // part[set][feature of the head]; a set's tensor follows from its group
  const int row = a.lanes * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (in0) part[set_in * row + o0 + i] = da[i];
    if (two) part[set_in * row + o1 + i] = db[i];
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

// dw[f] = the blocks' partial sums of feature f, in order within eight interleaved runs.
__global__ void __launch_bounds__(256) norm_weights_kernel(const float* part, int blocks, int D,
                                                           float* dq_w, float* dk_w) {
  __shared__ float run[8][32];
  const int f = blockIdx.x * 32 + (threadIdx.x & 31), k0 = threadIdx.x >> 5;
  grid_dependency_wait();
  float s = 0.f;
  if (f < 2 * D)
    for (int k = k0; k < blocks; k += 8) s += part[static_cast<int64_t>(k) * 2 * D + f];
  run[k0][threadIdx.x & 31] = s;
  __syncthreads();
  if (k0 || f >= 2 * D) return;
  for (int k = 1; k < 8; ++k) s += run[k][threadIdx.x];
  float* out = f < D ? dq_w : dk_w;
  if (out) out[f < D ? f : f - D] = s;
}

// Lanes per head, groups of heads.
void plan_groups(NormArgs* a, int heads) {
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

}  // namespace

cudaError_t launch_norm_rope(NormArgs a, bool interleaved, bool append, int64_t tokens,
                             cudaStream_t stream) {
  plan_groups(&a, kFwdHeads);
  const int64_t per_tok = static_cast<int64_t>(a.lanes) * a.r.n_groups;
  // thread indices fit 32 bits; a longer call goes in several launches
  const int64_t most = ((int64_t(1) << 31) - 1) / per_tok;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t n = tokens - t0 < most ? tokens - t0 : most;
    a.r.tok0 = t0;
    a.r.units = static_cast<uint32_t>(n * per_tok);
    const unsigned grid = static_cast<unsigned>((n * per_tok + kFwdThreads - 1) / kFwdThreads);
    launch_begin(16, stream);
    if (append) {
      if (interleaved) norm_rope_kernel<true, true><<<grid, kFwdThreads, 0, stream>>>(a);
      else norm_rope_kernel<false, true><<<grid, kFwdThreads, 0, stream>>>(a);
    } else {
      if (interleaved) norm_rope_kernel<true, false><<<grid, kFwdThreads, 0, stream>>>(a);
      else norm_rope_kernel<false, false><<<grid, kFwdThreads, 0, stream>>>(a);
    }
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
  plan_groups(&a, kBwdHeads);
  // a block for every 256 threads of work, at most kNormBwdBlocks; at least a walker for each group
  const int sets = kBwdThreads / a.lanes;
  const int64_t least = (static_cast<int64_t>(a.r.n_groups) + sets - 1) / sets;
  const int64_t work = tokens > (int64_t(1) << 32) ? int64_t(1) << 40 : tokens * a.r.n_groups;
  int64_t b = (work + sets - 1) / sets;
  if (b > kNormBwdBlocks) b = kNormBwdBlocks;
  return static_cast<int>(b < least ? least : b);
}

cudaError_t launch_norm_rope_bwd(NormArgs a, bool interleaved, float* dq_w, float* dk_w,
                                 cudaStream_t stream) {
  plan_groups(&a, kBwdHeads);
  const int blocks = norm_bwd_blocks(a.tokens, a.r.D, a.r.heads[0], a.r.heads[1]);
  launch_begin(16, stream);
  if (interleaved) norm_rope_bwd_kernel<true><<<blocks, kBwdThreads, 0, stream>>>(a);
  else norm_rope_bwd_kernel<false><<<blocks, kBwdThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  launch_end(16, stream);
  if (e != cudaSuccess || !a.part) return e;
  launch_begin(16, stream);
  e = launch_after(norm_weights_kernel, dim3((2 * a.r.D + 31) / 32), dim3(256), 0, stream, true,
                   static_cast<const float*>(a.part), blocks, a.r.D, dq_w, dk_w);
  launch_end(16, stream);
  return e;
}

}  // namespace upipe
