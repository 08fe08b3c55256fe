// attn_simple.cu -- attention of one new token with one warp per row.
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

// The new token of sequence b over its cache, one query head per warp.
__global__ void k_attn_token_simple(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(a.B) * a.Hq * a.Sq) return;
  const int i = row % a.Sq, h = row / a.Sq % a.Hq, b = row / a.Sq / a.Hq, g = h / a.group;
  const int Sk = min(max(a.lengths[b], 0), a.Sk);
  const int p = i + Sk - a.Sq;
  float q[kPer], o[kPer] = {}, x[kPer];
  load_row(a.q, b * a.sq[0] + i * a.sq[1] + h * a.sq[2], a.D, q);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < Sk; ++j) {
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
}

dim3 blocks(int64_t rows) { return dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_attn_token(const AttnArgs &a, cudaStream_t s) {
  return launch_pdl(k_attn_token_simple, blocks(int64_t(a.B) * a.Hq * a.Sq), dim3(32 * kWarps), 0, s, a);
}
}  // namespace lora
