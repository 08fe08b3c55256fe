// rotary.cu -- rotary positions of q and k (include/lora_rotary.h).
//
// One pass over q and k, bound by HBM (or by the launch where the tokens are
// few).  The angles are not read from a table: position * turns modulo 2^64
// is the angle's fraction of a turn, off by the position times 2^-65.  A block takes a few neighbouring
// tokens: its warps ask for their first heads, form the cosines and sines of
// all its tokens in shared memory meanwhile, and pass over the heads side by
// side, a lane keeping its place in the head.  Measured at 4096 tokens x 40
// heads of 128 in bf16, one pass: angles in registers of threads that turn
// eight heads 54 us; items divided among threads 20 us (300 instructions an
// item); a token to a warp 17 us, but in fp32 141 us where the warps of a
// block side by side take 120 us (5461 x 3 tokens x 48 heads), as here: 17 us
// (84 MB: 4.9 TB/s, much of it the launch's ramps), and 115 to 121 us (805 MB:
// 6.7 to 7.0 TB/s, a copy's bandwidth).
#include <cuda_bf16.h>

#include <cmath>

#include "host.h"
#include "lora_rotary.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kWarps = 8;

struct RotaryArgs {
  const void *in[2];
  void *out[2];
  int64_t is[2][3], os[2][3];
  const void *pos;
  int64_t ps[2];
  const uint64_t *turns;
  int64_t seq, all_tokens;
  int heads[2], dim, rot;
  // A head is rot_chunks chunks of VEC pairs, then chunks of 2 VEC copied
  // elements; the lanes take lane_heads heads at once (or 32 chunks of one).
  int rot_chunks, chunks, lane_heads;
  int groups[2];    // of lane_heads heads of q, of k
  int tokens;       // of a block
  int pos64;
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

// Cosines and sines of the VEC pairs of a lane's two vectors x and y.
template <int VEC>
struct Angles {
  float c[VEC], s[VEC];
};
// Turns the pairs (x[e], y[e]); with NEIGHBOURS those of neighbours in x, then
// in y (one element each: x and y are the pair).
template <class T, int VEC, bool NEIGHBOURS>
__device__ __forceinline__ void turn(Pack<T, VEC> &x, Pack<T, VEC> &y, const Angles<VEC> &a) {
  if constexpr (sizeof(T) == 2 && VEC == 8) {  // bf16, two elements a word
    uint32_t *xw = reinterpret_cast<uint32_t *>(x.v), *yw = reinterpret_cast<uint32_t *>(y.v);
    auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
    auto pack = [](float u, float v) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(u, v);
      return *reinterpret_cast<const uint32_t *>(&p);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = lo(xw[i]), x1 = hi(xw[i]), y0 = lo(yw[i]), y1 = hi(yw[i]);
      if constexpr (NEIGHBOURS) {
        const float cx = a.c[i], sx = a.s[i], cy = a.c[4 + i], sy = a.s[4 + i];
        xw[i] = pack(fmaf(x0, cx, -(x1 * sx)), fmaf(x1, cx, x0 * sx));
        yw[i] = pack(fmaf(y0, cy, -(y1 * sy)), fmaf(y1, cy, y0 * sy));
      } else {
        const float c0 = a.c[2 * i], s0 = a.s[2 * i], c1 = a.c[2 * i + 1], s1 = a.s[2 * i + 1];
        xw[i] = pack(fmaf(x0, c0, -(y0 * s0)), fmaf(x1, c1, -(y1 * s1)));
        yw[i] = pack(fmaf(y0, c0, x0 * s0), fmaf(y1, c1, x1 * s1));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      constexpr bool kWithin = NEIGHBOURS && VEC > 1;
      T &xe = !kWithin ? x.v[e] : 2 * e < VEC ? x.v[2 * e] : y.v[2 * e - VEC];
      T &ye = !kWithin ? y.v[e] : 2 * e + 1 < VEC ? x.v[2 * e + 1] : y.v[2 * e + 1 - VEC];
      const float xf = to_f(xe), yf = to_f(ye);
      xe = from_f<T>(fmaf(xf, a.c[e], -(yf * a.s[e])));
      ye = from_f<T>(fmaf(yf, a.c[e], xf * a.s[e]));
    }
  }
}

// The block's cosines and sines, an angle a thread.
template <class F>
__device__ __forceinline__ void form_angles(const RotaryArgs &a, float *shared, int tokens, F place) {
  const int half = a.rot / 2;
#pragma unroll 1
  for (int i = threadIdx.x; i < tokens * half; i += 32 * kWarps) {
    const int tk = i / half, pair = i - tk * half;
    unsigned b, s;
    place(tk, b, s);
    const int64_t at = b * a.ps[0] + s * a.ps[1];
    const uint64_t p = a.pos64 ? static_cast<uint64_t>(static_cast<const int64_t *>(a.pos)[at])
                               : static_cast<uint64_t>(static_cast<int64_t>(
                                     static_cast<const int32_t *>(a.pos)[at]));
    // the turn's fraction in [-1/2, 1/2) as a signed 64-bit fraction, rounded
    // once to 24 bits; sincospi takes half turns
    const int64_t frac = static_cast<int64_t>(p * a.turns[pair]);
    float sv, cv;
    sincospif(__ll2float_rn(frac) * 0x1p-63f, &sv, &cv);
    shared[tk * a.rot + pair] = cv * a.mag;
    shared[tk * a.rot + half + pair] = sv * (a.mag * a.sin_sign);
  }
}

template <class T, int VEC, bool NEIGHBOURS>  // pairs (2i, 2i + 1), else (i, i + rot / 2)
__global__ void __launch_bounds__(32 * kWarps, 4) k_rotary(const RotaryArgs a) {
  using P = Pack<T, VEC>;
  extern __shared__ float shared[];  // [tokens][cosines, sines][rot / 2]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, half = a.rot / 2;
  griddep_wait();
  griddep_launch_dependents();
  const unsigned token0 = blockIdx.x * static_cast<unsigned>(a.tokens);
  const int tokens = static_cast<int>(min(static_cast<unsigned>(a.tokens),
                                          static_cast<unsigned>(a.all_tokens) - token0));
  const unsigned seq = static_cast<unsigned>(a.seq), b0 = token0 / seq, s0 = token0 - b0 * seq;
  auto place = [&](int tk, unsigned &b, unsigned &s) {  // a block may cross sequences
    b = b0;
    s = s0 + tk;
    while (s >= seq) {
      s -= seq;
      ++b;
    }
  };
  const int groups = a.groups[0] + a.groups[1], units = tokens * groups;

  constexpr int U = VEC == 8 ? 2 : 4;  // head groups of a warp in flight
  bool formed = false;
  // chunks of a head beyond 32 take further passes
  for (int c0 = 0; c0 < a.chunks; c0 += 32) {
    const int lane_head = a.chunks > 32 ? 0 : lane / a.chunks;
    const int c = a.chunks > 32 ? c0 + lane : lane - lane_head * a.chunks;
    const bool turned = c < a.rot_chunks;
    // its two vectors: the same places in either layout of the pairs
    const bool apart = NEIGHBOURS && VEC == 1;
    const int copied = c - a.rot_chunks, copies = a.chunks - a.rot_chunks;
    const int e0 = !turned ? a.rot + VEC * copied : apart ? 2 * c : VEC * c;
    const int e1 = e0 + (!turned ? VEC * copies : apart ? 1 : half);
    const bool on = lane_head < a.lane_heads && c < a.chunks, two = on && e1 < a.dim;
    // the angles' places: NEIGHBOURS, those of x and of y a quarter of rot apart
    constexpr int kHalf = VEC > 1 ? VEC / 2 : 1;
    const int p0 = NEIGHBOURS && VEC > 1 ? e0 / 2 : c * VEC;
    const int p1 = NEIGHBOURS && VEC > 1 ? e1 / 2 : p0 + kHalf;

    int tk = 0, g = warp;  // unit: a head group of a token
    while (g >= groups) {
      g -= groups;
      ++tk;
    }
    for (int unit = warp; unit < units; unit += U * kWarps) {
      P x[U], y[U];
      T *dst[U];
      int token[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int t = g >= a.groups[0], h = (g - (t ? a.groups[0] : 0)) * a.lane_heads + lane_head;
        token[i] = on && h < a.heads[t] && tk < tokens ? tk : -1;
        if (token[i] >= 0) {
          unsigned b, s;
          place(tk, b, s);
          const T *src = static_cast<const T *>(a.in[t]) + b * a.is[t][0] + s * a.is[t][1] +
                         h * a.is[t][2];
          dst[i] = static_cast<T *>(a.out[t]) + b * a.os[t][0] + s * a.os[t][1] + h * a.os[t][2];
          x[i] = *reinterpret_cast<const P *>(src + e0);
          if (two) y[i] = *reinterpret_cast<const P *>(src + e1);
        }
        g += kWarps;
        while (g >= groups) {
          g -= groups;
          ++tk;
        }
      }
      if (!formed) {
        form_angles(a, shared, tokens, place);
        __syncthreads();
        formed = true;
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (token[i] >= 0) {
          if (turned) {
            const float *cosines = shared + token[i] * a.rot, *sines = cosines + half;
            Angles<VEC> angles;
            if constexpr (VEC > 1) {
              using H = Pack<float, kHalf>;
              *reinterpret_cast<H *>(angles.c) = *reinterpret_cast<const H *>(cosines + p0);
              *reinterpret_cast<H *>(angles.c + kHalf) = *reinterpret_cast<const H *>(cosines + p1);
              *reinterpret_cast<H *>(angles.s) = *reinterpret_cast<const H *>(sines + p0);
              *reinterpret_cast<H *>(angles.s + kHalf) = *reinterpret_cast<const H *>(sines + p1);
            } else {
              angles.c[0] = cosines[p0];
              angles.s[0] = sines[p0];
            }
            turn<T, VEC, NEIGHBOURS>(x[i], y[i], angles);
          }
          *reinterpret_cast<P *>(dst[i] + e0) = x[i];
          if (two) *reinterpret_cast<P *>(dst[i] + e1) = y[i];
        }
    }
    if (!formed) {  // a warp without a unit helps all the same
      form_angles(a, shared, tokens, place);
      __syncthreads();
      formed = true;
    }
  }
}

template <class T, int VEC>
cudaError_t launch_rotary(RotaryArgs &a, bool neighbours, bool copy_tail, int sms, cudaStream_t s) {
  a.rot_chunks = a.rot / 2 / VEC;
  a.chunks = a.rot_chunks + (copy_tail ? (a.dim - a.rot + 2 * VEC - 1) / (2 * VEC) : 0);
  a.lane_heads = a.chunks > 32 ? 1 : 32 / a.chunks;
  for (int t = 0; t < 2; ++t) a.groups[t] = (a.heads[t] + a.lane_heads - 1) / a.lane_heads;
  // Tokens of a block: some 32 KB of heads (in bf16, 10 KB a token, one token
  // takes 43 us where three to eight take 35 for 8192; in fp32, 24 KB a token,
  // eight take 131 us where one takes 121 for 16383), no more than 1024 angles,
  // and fewer while that would leave less than two blocks to an SM.
  const int64_t bytes = int64_t(a.heads[0] + a.heads[1]) * a.dim * sizeof(T);
  a.tokens = static_cast<int>(bytes > 32768 ? 1 : bytes * 8 < 32768 ? 8 : 32768 / bytes);
  while (a.tokens > 1 && (a.tokens * a.rot > 1024 || a.all_tokens < int64_t(a.tokens) * 2 * sms))
    a.tokens /= 2;
  const int64_t blocks = (a.all_tokens + a.tokens - 1) / a.tokens;
  return launch_pdl(neighbours ? k_rotary<T, VEC, true> : k_rotary<T, VEC, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps),
                    size_t(a.tokens) * a.rot * sizeof(float), s, a);
}

// The first 1152 binary places of 1 / (2 pi).
constexpr uint64_t kOverTwoPi[18] = {
    0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull,
    0x7f9458eaf7aef158ull, 0x6dc91b8e909374b8ull, 0x01924bba82746487ull,
    0x3f877ac72c4a69cfull, 0xba208d7d4baed121ull, 0x3a671c09ad17df90ull,
    0x4e64758e60d4ce7dull, 0x272117e2ef7e4a0eull, 0xc7fe25fff7816603ull,
    0xfbcbc462d6829b47ull, 0xdb4d9fb3c9f2c26dull, 0xd3d18fd9a797fa8bull,
    0x5d49eeb1faf97c5eull, 0xcf41ce7de294a4baull, 0x9afed7ec47e35742ull};
// Its 64 places from place `at` + 1 on (places before the first: 0).
uint64_t places(int at) {
  auto word = [](int i) { return i >= 0 && i < 18 ? kOverTwoPi[i] : uint64_t(0); };
  if (at <= -64) return 0;
  const int i = at < 0 ? -1 : at / 64, shift = at - 64 * i;  // 0 .. 63
  return shift == 0 ? word(i) : word(i) << shift | word(i + 1) >> (64 - shift);
}
// frac(w / 2 pi) * 2^64 to the nearest, for any finite w: w = m 2^e with whole m
// times those places of 1 / (2 pi) that count, as Payne and Hanek (1983) do it.
// (A quotient of doubles would be off by 2^-54 of a turn, times the position.)
uint64_t turns_of(double w) {
  int e;
  const double f = std::frexp(std::fabs(w), &e);  // in [1/2, 1)
  const uint64_t m = static_cast<uint64_t>(std::ldexp(f, 53));
  // T = m 2^(e - 53 + 64) / (2 pi) modulo 2^64: 64 places above 1 and 64 below
  const int s = e - 53 + 64;
  const uint64_t hi = places(s - 64), lo = places(s);
  const unsigned __int128 below = static_cast<unsigned __int128>(m) * lo + (uint64_t(1) << 63);
  const uint64_t t = m * hi + static_cast<uint64_t>(below >> 64);
  return w < 0 ? uint64_t(0) - t : t;
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
    turns[i] = turns_of(radians[i]);
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
    const int64_t entries[3] = {sh->batch, sh->seq, heads[t]};
    for (int j = 0; j < 3; ++j)
      if (entries[j] > 1 && os[t][j] == 0)
        return fail(LORA_ERR_INVALID_ARG, "%s_out is broadcast (stride 0)", name);
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
  a.heads[0] = sh->q_heads;
  a.heads[1] = sh->k_heads;
  a.dim = sh->dim;
  a.rot = sh->rot;
  a.mag = sh->magnitude;
  a.sin_sign = sh->inverse ? -1.f : 1.f;
  a.all_tokens = tokens;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_ROTARY, st, "rotary", [&] {
    if (dtype == LORA_BF16)
      return wide ? launch_rotary<__nv_bfloat16, 8>(a, sh->interleaved != 0, copy_tail, di.sms, st)
                  : launch_rotary<__nv_bfloat16, 1>(a, sh->interleaved != 0, copy_tail, di.sms, st);
    return wide ? launch_rotary<float, 4>(a, sh->interleaved != 0, copy_tail, di.sms, st)
                : launch_rotary<float, 1>(a, sh->interleaved != 0, copy_tail, di.sms, st);
  });
}

}  // extern "C"
