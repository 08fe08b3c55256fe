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
  // The ten rounds' keys (a Weyl sequence from the seed), made on the host: the
  // kernels' instructions take them straight from the argument block (adding
  // them up a thread cost a quarter of the dropout kernel's instructions).
  uint32_t keys[20] = {};
};
inline void drop_keys(DropArgs &d) {
  uint32_t k0 = static_cast<uint32_t>(d.seed), k1 = static_cast<uint32_t>(d.seed >> 32);
  for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    d.keys[2 * i] = k0;
    d.keys[2 * i + 1] = k1;
  }
}

// The seed and offset that count, read when the kernel runs.
struct DropNow {
  uint64_t seed;
  uint32_t offset;
};
__device__ __forceinline__ DropNow drop_now(const DropArgs &d) {
  if (d.state == nullptr) return {d.seed, d.offset};
  return {d.state[0], d.offset + static_cast<uint32_t>(d.state[1])};
}

// Philox4x32, ten rounds: each round multiplies two of the four words by the
// published constants and mixes the halves of the products with the others
// and with the round's key.
template <class Key>
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                          const Key &key) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = uint64_t(0xD2511F53u) * c0, q = uint64_t(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(q >> 32) ^ c1 ^ key(2 * i);
    c1 = static_cast<uint32_t>(q);
    c2 = static_cast<uint32_t>(p >> 32) ^ c3 ^ key(2 * i + 1);
    c3 = static_cast<uint32_t>(p);
  }
  return make_uint4(c0, c1, c2, c3);
}

// The four words of columns 4 b .. 4 b + 3 of a row.  (Where the seed comes from
// memory the keys are added up, in a function of its own: one copy of the code.)
static __device__ __noinline__ uint4 drop_words_of(uint64_t seed, uint32_t b, uint32_t lo, uint32_t hi,
                                            uint32_t offset) {
  const uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
  return philox10(b, lo, hi, offset, [&](int i) {
    return i & 1 ? k1 + 0xBB67AE85u * (i >> 1) : k0 + 0x9E3779B9u * (i >> 1);
  });
}
__device__ __forceinline__ uint4 drop_words(const DropArgs &d, const DropNow &now, uint32_t b,
                                            int64_t row) {
  const uint32_t lo = static_cast<uint32_t>(row), hi = static_cast<uint32_t>(uint64_t(row) >> 32);
  if (d.state == nullptr)
    return philox10(b, lo, hi, now.offset, [&](int i) { return d.keys[i]; });
  return drop_words_of(now.seed, b, lo, hi, now.offset);
}
__device__ __forceinline__ float drop1(const DropArgs &d, uint32_t word, float x) {
  return word >= d.threshold ? x * d.scale : 0.f;
}
// Columns 8 v .. 8 v + 7 of a row, in place.
__device__ __forceinline__ void drop8(const DropArgs &d, const DropNow &now, uint32_t v, int64_t row,
                                      float2 (&x)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 w = drop_words(d, now, 2 * v + h, row);
    const float2 a = __fmul2_rn(x[2 * h], make_float2(d.scale, d.scale));
    const float2 b = __fmul2_rn(x[2 * h + 1], make_float2(d.scale, d.scale));
    x[2 * h] = make_float2(w.x >= d.threshold ? a.x : 0.f, w.y >= d.threshold ? a.y : 0.f);
    x[2 * h + 1] = make_float2(w.z >= d.threshold ? b.x : 0.f, w.w >= d.threshold ? b.y : 0.f);
  }
}
__device__ __forceinline__ uint32_t word_of(const uint4 &w, uint32_t i) {
  const uint32_t lo = i & 1 ? w.y : w.x, hi = i & 1 ? w.w : w.z;
  return i & 2 ? hi : lo;
}

// ---- elements as pairs of fp32 (the packed fp32 instructions take two at a time) ----
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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
__device__ __forceinline__ uint32_t pack_pair(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 open_pair(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Keeps the compiler from working something out ahead of a loop over rows and
// holding it in registers all along (the weights as fp32, 32 addresses): they
// spilled, at more than the few instructions cost.
__device__ __forceinline__ uint32_t each_time(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}
__device__ __forceinline__ int each_time(int v) {
  asm volatile("" : "+r"(v));
  return v;
}
__device__ __forceinline__ float each_time(float v) {
  asm volatile("" : "+f"(v));
  return v;
}

// Eight elements as they lie in memory: aligned and side by side, or one by one.
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t u[4];
  __device__ __forceinline__ float2 pair(int i) const { return open_pair(u[i]); }
  __device__ __forceinline__ float2 again(int i) const { return open_pair(each_time(u[i])); }
  __device__ __forceinline__ void set(int i, float2 v) { u[i] = pack_pair(v); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void load1(int i, const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint16_t *>(p);
    u[i >> 1] = i & 1 ? __byte_perm(u[i >> 1], w, 0x5410) : w;  // (element 0 comes first)
  }
  __device__ __forceinline__ void store1(int i, __nv_bfloat16 *p) const {
    *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(i & 1 ? u[i >> 1] >> 16 : u[i >> 1]);
  }
};
template <>
struct Raw8<float> {
  float2 f[4];
  __device__ __forceinline__ float2 pair(int i) const { return f[i]; }
  __device__ __forceinline__ float2 again(int i) const { return f[i]; }
  __device__ __forceinline__ void set(int i, float2 v) { f[i] = v; }
  __device__ __forceinline__ void load(const float *p) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
  __device__ __forceinline__ void load1(int i, const float *p) { (i & 1 ? f[i >> 1].y : f[i >> 1].x) = *p; }
  __device__ __forceinline__ void store1(int i, float *p) const { *p = i & 1 ? f[i >> 1].y : f[i >> 1].x; }
};

// Host: the argument block of a checked description (dropout.cu).
lora_status_t drop_args(const lora_dropout_t *d, DropArgs &out);

}  // namespace lora
