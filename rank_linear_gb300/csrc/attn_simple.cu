// attn_simple.cu -- attention gradients and the one-token form with one warp per
// row, on CUDA cores.
#include <cuda_bf16.h>

#include <cmath>

#include "attn.h"
#include "host.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kWarps = 8, kPer = 4;  // a lane holds elements lane + 32 i of a head (dim <= 128)

using bf16 = __nv_bfloat16;

__device__ __forceinline__ void load_row(const void *p, int64_t off, int D, float (&r)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x % 32 + 32 * i;
    r[i] = e < D ? __bfloat162float(static_cast<const bf16 *>(p)[off + e]) : 0.f;
  }
}
__device__ __forceinline__ void store_row(void *p, int64_t off, int D, const float (&r)[kPer],
                                          float by) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x % 32 + 32 * i;
    if (e < D) static_cast<bf16 *>(p)[off + e] = __float2bfloat16_rn(r[i] * by);
  }
}
__device__ __forceinline__ float dot(const float (&a)[kPer], const float (&b)[kPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return s;
}

__device__ __forceinline__ bool visible(const AttnArgs &a, int b, int i, int j) {
  bool ok = !a.causal || j <= i + a.Sk - a.Sq || (a.prefix != nullptr && j < a.prefix[b]);
  if (a.q_docs != nullptr) {
    const int d = a.q_docs[b * a.qds + i];
    ok = ok && d >= 0 && d == a.k_docs[b * a.kds + j];
  }
  return ok;
}
// The score of z = q . k, and dc/dz.
__device__ __forceinline__ float score(const AttnArgs &a, int h, float z, int far, float &slope) {
  z *= a.scale;
  slope = 1.f;
  if (a.cap > 0.f) {
    const float t = tanhf(z / a.cap);
    z = a.cap * t;
    slope = 1.f - t * t;
  }
  if (a.slopes != nullptr) z -= a.slopes[h] * fabsf(static_cast<float>(far));
  return z;
}

// One query row per warp; TOKEN: the new token of sequence b over its cache.
template <bool TOKEN>
__global__ void k_attn_fwd_simple(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(a.B) * a.Hq * a.Sq) return;
  const int i = row % a.Sq, h = row / a.Sq % a.Hq, b = row / a.Sq / a.Hq, g = h / a.group;
  const int Sk = TOKEN ? min(max(a.lengths[b], 0), a.Sk) : a.Sk;
  const int p = i + Sk - a.Sq;
  float q[kPer], o[kPer] = {}, x[kPer];
  load_row(a.q, b * a.sq[0] + i * a.sq[1] + h * a.sq[2], a.D, q);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < Sk; ++j) {
    if (!TOKEN && !visible(a, b, i, j)) continue;
    load_row(a.k, b * a.sk[0] + j * a.sk[1] + g * a.sk[2], a.D, x);
    float d;
    const float s = score(a, h, dot(q, x), p - j, d);
    load_row(a.v, b * a.sv[0] + j * a.sv[1] + g * a.sv[2], a.D, x);
    const float m1 = fmaxf(m, s), keep = expf(m - m1), w = expf(s - m1);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = fmaf(o[e], keep, w * x[e]);
    m = m1;
  }
  store_row(a.o, b * a.so[0] + i * a.so[1] + h * a.so[2], a.D, o, l > 0.f ? 1.f / l : 0.f);
  if (!TOKEN && a.lse != nullptr && threadIdx.x % 32 == 0) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

// dq of one query row per warp, and delta = do . o.
__global__ void k_attn_dq_simple(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(a.B) * a.Hq * a.Sq) return;
  const int i = row % a.Sq, h = row / a.Sq % a.Hq, b = row / a.Sq / a.Hq, g = h / a.group;
  float q[kPer], e[kPer], x[kPer], dq[kPer] = {};
  load_row(a.q, b * a.sq[0] + i * a.sq[1] + h * a.sq[2], a.D, q);
  load_row(a.d_o, b * a.sdo[0] + i * a.sdo[1] + h * a.sdo[2], a.D, e);
  load_row(a.o, b * a.so[0] + i * a.so[1] + h * a.so[2], a.D, x);
  const float delta = dot(e, x), lse = a.lse[row];
  for (int j = 0; j < a.Sk; ++j) {
    if (!visible(a, b, i, j)) continue;
    float d;
    load_row(a.k, b * a.sk[0] + j * a.sk[1] + g * a.sk[2], a.D, x);
    const float s = score(a, h, dot(q, x), i + a.Sk - a.Sq - j, d);
    float y[kPer];
    load_row(a.v, b * a.sv[0] + j * a.sv[1] + g * a.sv[2], a.D, y);
    const float dz = expf(s - lse) * (dot(e, y) - delta) * d;
#pragma unroll
    for (int c = 0; c < kPer; ++c) dq[c] = fmaf(dz, x[c], dq[c]);
  }
  store_row(a.dq, b * a.sdq[0] + i * a.sdq[1] + h * a.sdq[2], a.D, dq, a.scale);
  if (threadIdx.x % 32 == 0) a.delta[row] = delta;
}

// dk and dv of one key row per warp.
__global__ void k_attn_dkv_simple(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(a.B) * a.Hk * a.Sk) return;
  const int j = row % a.Sk, g = row / a.Sk % a.Hk, b = row / a.Sk / a.Hk;
  float k[kPer], v[kPer], x[kPer], y[kPer], dk[kPer] = {}, dv[kPer] = {};
  load_row(a.k, b * a.sk[0] + j * a.sk[1] + g * a.sk[2], a.D, k);
  load_row(a.v, b * a.sv[0] + j * a.sv[1] + g * a.sv[2], a.D, v);
  for (int h = g * a.group; h < (g + 1) * a.group; ++h)
    for (int i = 0; i < a.Sq; ++i) {
      if (!visible(a, b, i, j)) continue;
      float d;
      load_row(a.q, b * a.sq[0] + i * a.sq[1] + h * a.sq[2], a.D, x);
      load_row(a.d_o, b * a.sdo[0] + i * a.sdo[1] + h * a.sdo[2], a.D, y);
      const float s = score(a, h, dot(x, k), i + a.Sk - a.Sq - j, d);
      const int64_t r = (static_cast<int64_t>(b) * a.Hq + h) * a.Sq + i;
      const float p = expf(s - a.lse[r]);
      const float dz = p * (dot(y, v) - a.delta[r]) * d;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        dk[c] = fmaf(dz, x[c], dk[c]);
        dv[c] = fmaf(p, y[c], dv[c]);
      }
    }
  store_row(a.dk, b * a.sdk[0] + j * a.sdk[1] + g * a.sdk[2], a.D, dk, a.scale);
  store_row(a.dv, b * a.sdv[0] + j * a.sdv[1] + g * a.sdv[2], a.D, dv, 1.f);
}

dim3 blocks(int64_t rows) { return dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_attn_token(const AttnArgs &a, cudaStream_t s) {
  return launch_pdl(k_attn_fwd_simple<true>, blocks(int64_t(a.B) * a.Hq * a.Sq), dim3(32 * kWarps), 0, s, a);
}
cudaError_t launch_attn_dq(const AttnArgs &a, cudaStream_t s) {
  return launch_pdl(k_attn_dq_simple, blocks(int64_t(a.B) * a.Hq * a.Sq), dim3(32 * kWarps), 0, s, a);
}
cudaError_t launch_attn_dkv(const AttnArgs &a, cudaStream_t s) {
  return launch_pdl(k_attn_dkv_simple, blocks(int64_t(a.B) * a.Hk * a.Sk), dim3(32 * kWarps), 0, s, a);
}

}  // namespace lora
