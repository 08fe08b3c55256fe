// rotary.cu -- rotary positions of q and k (include/lora_rotary.h).
//
// One pass over q and k, bound by HBM (or by the launch where the tokens are
// few).  The angles are not read from a table: position * turns modulo 2^64
// is the angle's exact fraction of a turn, and a thread keeps the cosines and
// sines of its VEC pairs in registers for all the heads it turns, so that
// their cost is spread over kHeads heads.
#include <cuda_bf16.h>

#include <cmath>

#include "host.h"
#include "lora_rotary.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
  const void *in[2];
  void *out[2];
  int64_t is[2][3], os[2][3];
  const void *pos;
  int64_t ps[2];
  const uint64_t *turns;
  int64_t seq, items;  // items: tokens * head groups * chunks
  int q_heads, heads, dim, rot;
  int rot_chunks, chunks;  // chunks of VEC pairs; then of 2 VEC copied elements
  int groups, per;         // head groups of `per` heads
  int interleaved, pos64;
  float mag, sin_sign;
};

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

// A thread's item: one chunk (VEC pairs, or up to 2 VEC copied elements) of
// `per` heads of one token.  A chunk is two vectors at offsets e0 and e1.
template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryArgs a) {
  using P = Pack<T, VEC>;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= a.items) return;
  const int c = static_cast<int>(item % a.chunks);
  const int64_t rest = item / a.chunks;
  const int group = static_cast<int>(rest % a.groups);
  const int64_t token = rest / a.groups;
  const int64_t b = token / a.seq, s = token % a.seq;

  const bool turn = c < a.rot_chunks;
  int e0, e1;
  bool two = true;
  float cs[VEC], sn[VEC];
  if (turn) {
    const int i0 = c * VEC;
    e0 = a.interleaved ? 2 * i0 : i0;
    e1 = a.interleaved ? 2 * i0 + VEC : i0 + a.rot / 2;
    const int64_t at = b * a.ps[0] + s * a.ps[1];
    const uint64_t p = a.pos64 ? static_cast<uint64_t>(static_cast<const int64_t *>(a.pos)[at])
                               : static_cast<uint64_t>(static_cast<int64_t>(
                                     static_cast<const int32_t *>(a.pos)[at]));
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // the turn's fraction in [-1/2, 1/2) as a signed 64-bit fraction,
      // rounded once to 24 bits; sincospi takes half turns
      const int64_t frac = static_cast<int64_t>(p * __ldg(a.turns + i0 + e));
      float sv, cv;
      sincospif(__ll2float_rn(frac) * 0x1p-63f, &sv, &cv);
      cs[e] = cv * a.mag;
      sn[e] = sv * (a.mag * a.sin_sign);
    }
  } else {
    e0 = a.rot + (c - a.rot_chunks) * 2 * VEC;
    e1 = e0 + VEC;
    two = e1 < a.dim;
  }

  const int h0 = group * a.per, h1 = min(h0 + a.per, a.heads);
  constexpr int U = 4;  // heads in flight
  for (int hb = h0; hb < h1; hb += U) {
    P x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u;
      if (h < h1) {
        const int t = h >= a.q_heads;
        const int64_t off =
            b * a.is[t][0] + s * a.is[t][1] + (h - (t ? a.q_heads : 0)) * a.is[t][2];
        const T *src = static_cast<const T *>(a.in[t]) + off;
        x[u] = *reinterpret_cast<const P *>(src + e0);
        if (two) y[u] = *reinterpret_cast<const P *>(src + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u;
      if (h < h1) {
        if (turn) {
          float f[2 * VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            f[e] = to_f(x[u].v[e]);
            f[VEC + e] = to_f(y[u].v[e]);
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            // half: (x[e], y[e]); interleaved: neighbours of the 2 VEC run
            float &p = a.interleaved ? f[2 * e] : f[e];
            float &q = a.interleaved ? f[2 * e + 1] : f[VEC + e];
            const float px = p, qx = q;
            p = px * cs[e] - qx * sn[e];
            q = qx * cs[e] + px * sn[e];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x[u].v[e] = from_f<T>(f[e]);
            y[u].v[e] = from_f<T>(f[VEC + e]);
          }
        }
        const int t = h >= a.q_heads;
        const int64_t off =
            b * a.os[t][0] + s * a.os[t][1] + (h - (t ? a.q_heads : 0)) * a.os[t][2];
        T *dst = static_cast<T *>(a.out[t]) + off;
        *reinterpret_cast<P *>(dst + e0) = x[u];
        if (two) *reinterpret_cast<P *>(dst + e1) = y[u];
      }
    }
  }
}

template <class T, int VEC>
cudaError_t launch_rotary(RotaryArgs &a, int64_t tokens, bool copy_tail, int sms, cudaStream_t s) {
  a.rot_chunks = a.rot / 2 / VEC;
  a.chunks = a.rot_chunks + (copy_tail ? (a.dim - a.rot + 2 * VEC - 1) / (2 * VEC) : 0);
  // heads per thread: 8 to spread the angles' cost, fewer while that would
  // leave SMs without a block
  a.per = 8;
  while (a.per > 1 &&
         tokens * a.chunks * ((a.heads + a.per - 1) / a.per) < int64_t(sms) * kThreads)
    a.per /= 2;
  a.groups = (a.heads + a.per - 1) / a.per;
  a.items = tokens * a.groups * a.chunks;
  const int64_t blocks = (a.items + kThreads - 1) / kThreads;
  return launch_pdl(k_rotary<T, VEC>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, a);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_rotary_turns(const double *radians, int n, uint64_t *turns) {
  clear_error();
  if (n < 0) return fail(LORA_ERR_INVALID_ARG, "n = %d is negative", n);
  if (n > 0 && (radians == nullptr || turns == nullptr))
    return fail(LORA_ERR_INVALID_ARG, "radians or turns is NULL");
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(radians[i]))
      return fail(LORA_ERR_INVALID_ARG, "radians[%d] is not finite", i);
    double t = radians[i] / 6.283185307179586476925286766559;
    t -= std::floor(t);
    const double v = std::ldexp(t, 64);  // t == 1.0 (rounded up) is a whole turn: 0
    turns[i] = v >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(v);
  }
  return LORA_OK;
}

lora_status_t lora_rotary(const lora_rotary_t *sh, const void *q, const void *k,
                          const void *positions, const uint64_t *turns, lora_dtype_t dtype,
                          void *q_out, void *k_out, void *stream) {
  clear_error();
  if (sh == nullptr) return fail(LORA_ERR_INVALID_ARG, "shape is NULL");
  if (dtype != LORA_BF16 && dtype != LORA_FP32)
    return fail(LORA_ERR_INVALID_ARG, "dtype %d is not LORA_BF16 or LORA_FP32", int(dtype));
  const int64_t kMax = int64_t(1) << 31;
  if (sh->batch < 0 || sh->seq < 0 || sh->q_heads < 0 || sh->k_heads < 0)
    return fail(LORA_ERR_INVALID_ARG, "batch, seq or a number of heads is negative");
  if (sh->batch > kMax || sh->seq > kMax || sh->batch * sh->seq > kMax || sh->q_heads > 65536 ||
      sh->k_heads > 65536)
    return fail(LORA_ERR_UNSUPPORTED, "more than 2^31 tokens or 65536 heads");
  if (sh->dim < 2 || sh->dim > 1024 || sh->rot < 2 || sh->rot > sh->dim || sh->rot % 2 != 0)
    return fail(LORA_ERR_INVALID_ARG, "rot = %d of dim = %d: rot must be even, 2 <= rot <= dim <= 1024",
                sh->rot, sh->dim);
  if ((sh->interleaved | 1) != 1 || (sh->inverse | 1) != 1)
    return fail(LORA_ERR_INVALID_ARG, "interleaved and inverse are 0 or 1");
  if (sh->position_bits != 32 && sh->position_bits != 64)
    return fail(LORA_ERR_INVALID_ARG, "position_bits = %d is not 32 or 64", sh->position_bits);
  if (!std::isfinite(sh->magnitude)) return fail(LORA_ERR_INVALID_ARG, "magnitude is not finite");
  const int64_t tokens = sh->batch * sh->seq;
  if (tokens == 0 || sh->q_heads + sh->k_heads == 0) return LORA_OK;

  const int es = dtype == LORA_BF16 ? 2 : 4;
  auto aligned = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (positions == nullptr || turns == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "positions or turns is NULL");
  if (!aligned(positions, sh->position_bits / 8) || !aligned(turns, 8))
    return fail(LORA_ERR_INVALID_ARG, "positions or turns is not aligned to its type");
  RotaryArgs a = {};
  const void *in[2] = {q, k};
  void *out[2] = {q_out, k_out};
  const int64_t *is[2] = {sh->q_in, sh->k_in}, *os[2] = {sh->q_out, sh->k_out};
  const int heads[2] = {sh->q_heads, sh->k_heads};
  const int vec = 16 / es;
  bool wide = sh->rot % (2 * vec) == 0 && sh->dim % vec == 0, copy_tail = false;
  for (int t = 0; t < 2; ++t) {
    if (heads[t] == 0) continue;
    const char *name = t == 0 ? "q" : "k";
    if (in[t] == nullptr || out[t] == nullptr)
      return fail(LORA_ERR_INVALID_ARG, "%s or %s_out is NULL", name, name);
    if (!aligned(in[t], es) || !aligned(out[t], es))
      return fail(LORA_ERR_INVALID_ARG, "%s or %s_out is not aligned to its type", name, name);
    bool same = in[t] == out[t];
    wide = wide && aligned(in[t], 16) && aligned(out[t], 16);
    for (int j = 0; j < 3; ++j) {
      a.is[t][j] = is[t][j];
      a.os[t][j] = os[t][j];
      same = same && is[t][j] == os[t][j];
      wide = wide && is[t][j] % vec == 0 && os[t][j] % vec == 0;
    }
    if (in[t] == out[t] && !same)
      return fail(LORA_ERR_INVALID_ARG, "%s_out is %s with other strides", name, name);
    copy_tail = copy_tail || (!same && sh->rot < sh->dim);
    a.in[t] = in[t];
    a.out[t] = out[t];
  }
  a.pos = positions;
  a.ps[0] = sh->position[0];
  a.ps[1] = sh->position[1];
  a.pos64 = sh->position_bits == 64;
  a.turns = turns;
  a.seq = sh->seq;
  a.q_heads = sh->q_heads;
  a.heads = sh->q_heads + sh->k_heads;
  a.dim = sh->dim;
  a.rot = sh->rot;
  a.interleaved = sh->interleaved;
  a.mag = sh->magnitude;
  a.sin_sign = sh->inverse ? -1.f : 1.f;
  // at most one item per pair (or copied pair) and head
  if (tokens * a.heads > (int64_t(1) << 31) * kThreads / (sh->dim + 2))
    return fail(LORA_ERR_UNSUPPORTED, "too many elements for one launch");
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_ROTARY, st, "rotary", [&] {
    if (dtype == LORA_BF16)
      return wide ? launch_rotary<__nv_bfloat16, 8>(a, tokens, copy_tail, di.sms, st)
                  : launch_rotary<__nv_bfloat16, 1>(a, tokens, copy_tail, di.sms, st);
    return wide ? launch_rotary<float, 4>(a, tokens, copy_tail, di.sms, st)
                : launch_rotary<float, 1>(a, tokens, copy_tail, di.sms, st);
  });
}

}  // extern "C"
