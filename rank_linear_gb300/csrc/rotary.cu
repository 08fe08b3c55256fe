// rotary.cu -- rotary positions of q and k (include/lora_rotary.h).
//
// One pass over q and k, bound by HBM (or by the launch where the tokens are
// few).  The angles are not read from a table: position * turns modulo 2^64
// is the angle's exact fraction of a turn.  A block takes a few tokens: it
// asks for its first vectors, turns the positions into cosines and sines in
// shared memory meanwhile (once for all heads), and passes over its heads in
// items of two vectors.  (With the angles in each thread's registers for
// eight heads, 124 registers and little in flight: 54 us instead of 17 at
// 4096 tokens x 40 heads of 128, bf16.)
#include <cuda_bf16.h>

#include <cmath>

#include "host.h"
#include "lora_rotary.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;

// n / d for n, d < 2^16: mul = ceil(2^32 / d).
struct Divide {
  uint32_t d, mul;
  __device__ __forceinline__ int by(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul));
  }
};
Divide divide(int d) {
  return {static_cast<uint32_t>(d),
          static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / static_cast<uint64_t>(d))};
}

struct RotaryArgs {
  const void *in[2];
  void *out[2];
  int64_t is[2][3], os[2][3];
  const void *pos;
  int64_t ps[2];
  const uint64_t *turns;
  int64_t seq, all_tokens;
  int q_heads, heads, dim, rot;
  int rot_chunks, chunks;  // of a head: VEC pairs each; then 2 VEC copied elements each
  int tokens;              // of a block
  Divide by_chunks, by_heads;
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

// An item: one chunk (VEC pairs, or up to 2 VEC copied elements) of one head
// of one token, as two vectors.
template <class T, int VEC, bool NEIGHBOURS>  // pairs (2i, 2i + 1), else (i, i + rot / 2)
__global__ void __launch_bounds__(kThreads, 4) k_rotary(const RotaryArgs a) {
  using P = Pack<T, VEC>;
  extern __shared__ float angles[];  // [tokens][2][rot / 2]: cosines, sines
  griddep_wait();
  griddep_launch_dependents();
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int tokens = static_cast<int>(
      a.all_tokens - token0 < a.tokens ? a.all_tokens - token0 : a.tokens);
  const int half = a.rot / 2, items = tokens * a.heads * a.chunks;
  const int64_t b0 = token0 / a.seq, s0 = token0 - b0 * a.seq;

  constexpr int U = 2;  // items of a thread in flight
  bool angles_there = false;
  for (int base = threadIdx.x; base - static_cast<int>(threadIdx.x) < items; base += U * kThreads) {
    P x[U], y[U];
    T *dst[U];
    int chunk[U], tok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int item = base + u * kThreads;
      chunk[u] = -1;
      if (item < items) {
        const int row = a.by_chunks.by(item), c = item - row * a.chunks;
        const int tk = a.by_heads.by(row), h = row - tk * a.heads;
        int64_t b = b0, s = s0 + tk;
        while (s >= a.seq) {  // a block may cross into the next sequences
          s -= a.seq;
          ++b;
        }
        const int t = h >= a.q_heads, ht = h - (t ? a.q_heads : 0);
        const T *src = static_cast<const T *>(a.in[t]) + b * a.is[t][0] + s * a.is[t][1] +
                       ht * a.is[t][2];
        dst[u] = static_cast<T *>(a.out[t]) + b * a.os[t][0] + s * a.os[t][1] + ht * a.os[t][2];
        chunk[u] = c;
        tok[u] = tk;
        const bool turn = c < a.rot_chunks;
        const int e0 = !turn ? a.rot + (c - a.rot_chunks) * 2 * VEC
                             : NEIGHBOURS ? 2 * VEC * c : VEC * c;
        const int e1 = turn && !NEIGHBOURS ? e0 + half : e0 + VEC;
        x[u] = *reinterpret_cast<const P *>(src + e0);
        if (turn || e1 < a.dim) y[u] = *reinterpret_cast<const P *>(src + e1);
      }
    }
    if (!angles_there) {
      for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int tk = i / half, pair = i - tk * half;
        int64_t b = b0, s = s0 + tk;
        while (s >= a.seq) {
          s -= a.seq;
          ++b;
        }
        const int64_t at = b * a.ps[0] + s * a.ps[1];
        const uint64_t p = a.pos64 ? static_cast<uint64_t>(static_cast<const int64_t *>(a.pos)[at])
                                   : static_cast<uint64_t>(static_cast<int64_t>(
                                         static_cast<const int32_t *>(a.pos)[at]));
        // the turn's fraction in [-1/2, 1/2) as a signed 64-bit fraction,
        // rounded once to 24 bits; sincospi takes half turns
        const int64_t frac = static_cast<int64_t>(p * a.turns[pair]);
        float sv, cv;
        sincospif(__ll2float_rn(frac) * 0x1p-63f, &sv, &cv);
        angles[(2 * tk) * half + pair] = cv * a.mag;
        angles[(2 * tk + 1) * half + pair] = sv * (a.mag * a.sin_sign);
      }
      __syncthreads();
      angles_there = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = chunk[u];
      if (c < 0) continue;
      const bool turn = c < a.rot_chunks;
      const int e0 = !turn ? a.rot + (c - a.rot_chunks) * 2 * VEC
                           : NEIGHBOURS ? 2 * VEC * c : VEC * c;
      const int e1 = turn && !NEIGHBOURS ? e0 + half : e0 + VEC;
      if (turn) {
        const float *cs = angles + 2 * tok[u] * half + VEC * c, *sn = cs + half;
        const Pack<float, VEC> cv = *reinterpret_cast<const Pack<float, VEC> *>(cs);
        const Pack<float, VEC> sv = *reinterpret_cast<const Pack<float, VEC> *>(sn);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          // NEIGHBOURS: element 2e and 2e + 1 of the run x, y
          T &xe = !NEIGHBOURS ? x[u].v[e] : 2 * e < VEC ? x[u].v[2 * e] : y[u].v[2 * e - VEC];
          T &ye = !NEIGHBOURS       ? y[u].v[e]
                  : 2 * e + 1 < VEC ? x[u].v[2 * e + 1]
                                    : y[u].v[2 * e + 1 - VEC];
          const float xf = to_f(xe), yf = to_f(ye);
          xe = from_f<T>(fmaf(xf, cv.v[e], -(yf * sv.v[e])));
          ye = from_f<T>(fmaf(yf, cv.v[e], xf * sv.v[e]));
        }
      }
      *reinterpret_cast<P *>(dst[u] + e0) = x[u];
      if (turn || e1 < a.dim) *reinterpret_cast<P *>(dst[u] + e1) = y[u];
    }
  }
}

template <class T, int VEC>
cudaError_t launch_rotary(RotaryArgs &a, bool copy_tail, int sms, cudaStream_t s) {
  a.rot_chunks = a.rot / 2 / VEC;
  a.chunks = a.rot_chunks + (copy_tail ? (a.dim - a.rot + 2 * VEC - 1) / (2 * VEC) : 0);
  // tokens of a block: up to 4, fewer while that would leave SMs without a
  // block or a block with more items than its 16-bit divisions take
  a.tokens = 4;
  while (a.tokens > 1 && (a.all_tokens < int64_t(a.tokens) * 2 * sms ||
                          int64_t(a.tokens) * a.heads * a.chunks > 65535))
    a.tokens /= 2;
  if (int64_t(a.heads) * a.chunks > 65535) return cudaErrorInvalidValue;
  a.by_chunks = divide(a.chunks);
  a.by_heads = divide(a.heads);
  const int64_t blocks = (a.all_tokens + a.tokens - 1) / a.tokens;
  return launch_pdl(a.interleaved ? k_rotary<T, VEC, true> : k_rotary<T, VEC, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                    size_t(a.tokens) * a.rot * sizeof(float), s, a);
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
  if (sh->batch >= kMax || sh->seq >= kMax || sh->batch * sh->seq >= kMax || sh->q_heads > 32768 ||
      sh->k_heads > 32768)
    return fail(LORA_ERR_UNSUPPORTED, "2^31 tokens or more, or over 32768 heads");
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
  a.all_tokens = tokens;
  // a token's items, one pair (or copied pair) each at the most
  if (int64_t(a.heads) * ((sh->dim + 1) / 2 + 1) > 65535)
    return fail(LORA_ERR_UNSUPPORTED, "%d heads of %d: too many elements in a token", a.heads,
                sh->dim);
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_ROTARY, st, "rotary", [&] {
    if (dtype == LORA_BF16)
      return wide ? launch_rotary<__nv_bfloat16, 8>(a, copy_tail, di.sms, st)
                  : launch_rotary<__nv_bfloat16, 1>(a, copy_tail, di.sms, st);
    return wide ? launch_rotary<float, 4>(a, copy_tail, di.sms, st)
                : launch_rotary<float, 1>(a, copy_tail, di.sms, st);
  });
}

}  // extern "C"
