// dropout.cuh -- the counter-based mask of include/lora_dropout.h, shared by
// the dropout and the norm kernels, and vectors of eight elements.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "lora_dropout.h"

namespace lora {

struct DropArgs {
  uint32_t threshold = 0;  // T; 0 keeps everything
  float scale = 1.f;       // 2^32 / (2^32 - T)
  uint64_t seed = 0;
  uint32_t offset = 0;
  const uint64_t *state = nullptr;
};

// The seed and offset that count, read when the kernel runs.
__device__ __forceinline__ void drop_resolve(DropArgs &d) {
  if (d.state != nullptr) {
    d.seed = d.state[0];
    d.offset += static_cast<uint32_t>(d.state[1]);
  }
}

// Philox4x32, ten rounds: each round multiplies two of the four words by the
// published constants and mixes the halves of the products with the others
// and with a key that advances by a Weyl sequence.
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                          uint64_t key) {
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = uint64_t(0xD2511F53u) * c0, q = uint64_t(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(q >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(q);
    c2 = static_cast<uint32_t>(p >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The four words of columns 4 b .. 4 b + 3 of a row.
__device__ __forceinline__ uint4 drop_words(const DropArgs &d, uint32_t b, int64_t row) {
  return philox10(b, static_cast<uint32_t>(row), static_cast<uint32_t>(uint64_t(row) >> 32),
                  d.offset, d.seed);
}
// Columns 8 v .. 8 v + 7 of a row, in place.
__device__ __forceinline__ void drop8(const DropArgs &d, uint32_t v, int64_t row, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = drop_words(d, 2 * v + h, row);
    x[4 * h + 0] = w.x >= d.threshold ? x[4 * h + 0] * d.scale : 0.f;
    x[4 * h + 1] = w.y >= d.threshold ? x[4 * h + 1] * d.scale : 0.f;
    x[4 * h + 2] = w.z >= d.threshold ? x[4 * h + 2] * d.scale : 0.f;
    x[4 * h + 3] = w.w >= d.threshold ? x[4 * h + 3] * d.scale : 0.f;
  }
}
__device__ __forceinline__ uint32_t word_of(const uint4 &w, uint32_t i) {
  const uint32_t lo = i & 1 ? w.y : w.x, hi = i & 1 ? w.w : w.z;
  return i & 2 ? hi : lo;
}

// ---- elements as fp32 ----
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight consecutive elements as they lie in memory (16-byte aligned).
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Raw8<float> {
  float4 a, b;
};
__device__ __forceinline__ void load_raw(const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
  r.a = *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void load_raw(const float *p, Raw8<float> &r) {
  r.a = reinterpret_cast<const float4 *>(p)[0];
  r.b = reinterpret_cast<const float4 *>(p)[1];
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
  const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw8<float> &r, float (&v)[8]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
  v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Host: the argument block of a checked description (dropout.cu).
lora_status_t drop_args(const lora_dropout_t *d, DropArgs &out);

}  // namespace lora
