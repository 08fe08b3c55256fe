// loss.cuh -- what the kernels of the large-vocabulary loss share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace lora {

constexpr int kLossTileM = 256, kLossTileN = 512;  // of a CTA pair
constexpr int kLossBlockK = 64;                    // length of a block of the products
constexpr int kLossPiece = 128;                    // columns of one partial sum
constexpr int kLossMaxPairs = 76;                  // of 152 SMs
constexpr size_t kLossSlotFloats = size_t(kLossTileM) * kLossTileN;
constexpr int kLossSlots = 2 * kLossMaxPairs;      // partial tiles of the second product

// What the device finds out about the call's tokens.
struct LossHead {
  int live;       // tokens that count
  float divisor;  // what the weights are divided by
};

// A partial sum of exp2(u - up), up a whole number > 0 where some u exceeds
// kLossFar (else 0).
struct LossPart {
  float sum, up;
};
constexpr float kLossFar = 64.f;

// How the pairs share the second product's tiles (rows x dim, K = vocab in kb
// blocks of 64).  Tiles fill whole rounds of the pairs; of the rest,
//   at most half as many as pairs: each is cut into `cuts` equal ranges of K,
//   more: the pairs without a tile take the last blocks, from `from` on, of
//         `each` tiles (at most) apiece, so that all end together.
// Ranges leave fp32 partial tiles, which are joined in their order.
struct LossShare {
  int tiles, pairs, whole, rest, cuts, from, each;
};
__host__ __device__ inline LossShare loss_share(int tiles, int pairs, int kb) {
  LossShare s = {tiles, pairs, tiles / pairs * pairs, tiles % pairs, 1, kb, 0};
  if (s.rest == 0) return s;
  const int least = 16;  // blocks of a range: below, writing and joining it costs as much
  if (2 * s.rest <= pairs) {
    const int most = kb / least;
    s.cuts = pairs / s.rest < most ? pairs / s.rest : most;
    if (s.cuts < 1) s.cuts = 1;
    return s;
  }
  const int spare = pairs - s.rest;
  if (spare == 0) return s;
  const int each = (s.rest + spare - 1) / spare;
  const int tail = kb / (each + 1);
  if (each > 8 || tail < least) return s;
  s.each = each;
  s.from = kb - tail;
  return s;
}
// Whether tile `tile` is left in ranges, how many, and where their slots start.
__host__ __device__ inline int loss_ranges(const LossShare &s, int tile, int &slot) {
  const int rel = tile - s.whole;
  if (rel < 0) return 1;
  const int n = s.each > 0 ? 2 : s.cuts;
  slot = rel * n;
  return n;
}
// Item `i` of a pair: the tile, its range of blocks and the slot for it (-1: the
// whole tile).  False after the last.
__host__ __device__ inline bool loss_item(const LossShare &s, int pair, int i, int kb, int &tile,
                                          int &lo, int &hi, int &slot) {
  const int rounds = s.whole / s.pairs;
  lo = 0;
  hi = kb;
  slot = -1;
  if (i < rounds) {
    tile = i * s.pairs + pair;
    return true;
  }
  i -= rounds;
  if (s.each > 0) {
    if (pair < s.rest) {
      tile = s.whole + pair;
      hi = s.from;
      slot = 2 * pair;
      return i == 0;
    }
    const int rel = pair - s.rest + i * (s.pairs - s.rest);
    tile = s.whole + rel;
    lo = s.from;
    slot = 2 * rel + 1;
    return rel < s.rest;
  }
  if (i > 0 || pair >= s.rest * s.cuts) return false;
  const int rel = pair % s.rest, c = pair / s.rest;
  tile = s.whole + rel;
  lo = static_cast<int>(int64_t(c) * kb / s.cuts);
  hi = static_cast<int>(int64_t(c + 1) * kb / s.cuts);
  if (s.cuts > 1) slot = rel * s.cuts + c;
  return true;
}
// The first product's items: whole tiles in rounds of the pairs; where at most half
// the pairs have one in the last round, they are taken as two halves of 256 columns
// each.  half: 0 or 1, or -1 for a whole tile.
__host__ __device__ inline bool loss_first_item(int tiles, int pairs, int pair, int i, int &tile,
                                                int &half) {
  const int rounds = tiles / pairs, rest = tiles % pairs;
  half = -1;
  if (i < rounds || 2 * rest > pairs) {
    tile = i * pairs + pair;
    return tile < tiles;
  }
  tile = rounds * pairs + (pair >> 1);
  half = pair & 1;
  return i == rounds && pair < 2 * rest;
}
// Tiles of a round share few panels: the rows vary fastest, in groups.
__host__ __device__ inline void loss_tile(int tile, int m_pairs, int n_tiles, int group, int &mp,
                                          int &nb) {
  const int per = group * n_tiles, g = tile / per, first = g * group;
  const int gm = group < m_pairs - first ? group : m_pairs - first, local = tile - g * per;
  mp = first + local % gm;
  nb = local / gm;
}

struct LossGemm {
  CUtensorMap a, b, e;  // operands; e: the strip of exponentials (written)
  const LossHead *head = nullptr;
  int first = 0, strip = 0;  // the strip's first counted token, and its most
  int n = 0, k = 0;          // columns of the result, length of the products
  int group = 8;
  float cap = 0.f;
  // first product
  const float *ref = nullptr;  // reference of each row, in units of log2
  const int *target = nullptr;
  LossPart *parts = nullptr;   // [piece][strip]
  float *own = nullptr;        // the target's u of each row
  // second product
  const float *scale = nullptr;  // of each row
  const int *place = nullptr;    // where each row of the strip goes
  __nv_bfloat16 *out = nullptr;
  int64_t ldo = 0;
  float *slots = nullptr;
  unsigned *dev_status = nullptr;
};
// kind 0: sums only, 1: sums and exponentials, 2: the second product.
cudaError_t launch_loss_gemm(int kind, const LossGemm &g, int pairs, cudaStream_t s);
// CTA pairs that are resident at once (at most kLossMaxPairs).
int loss_pairs(int num_sms);

__device__ __forceinline__ uint32_t loss_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// c(z) = cap tanh(z / cap) and c'(z), to a few 2^-23 of their size at any cap:
// for |z| <= cap / 4 the series of tanh (its next term is below 2^-26), beyond
// from e = exp(-2 |z| / cap): tanh = (1 - e) / (1 + e), 1 - tanh^2 = 4 e / (1 + e)^2.
__device__ __forceinline__ float loss_cap(float z, float cap, float inv_cap, float &slope) {
  const float x = z * inv_cap, y = x * x;
  float p = fmaf(y, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(p, y, 2.f / 15.f);
  p = fmaf(p, y, -1.f / 3.f);
  p = fmaf(p, y, 1.f);
  const float near = x * p;
  const float e = exp2f(fabsf(x) * -2.885390082f), r = __fdividef(1.f, 1.f + e);
  const bool far = y > 0.0625f;
  const float t = far ? copysignf((1.f - e) * r, x) : near;
  slope = far ? 4.f * e * r * r : fmaf(-near, near, 1.f);
  return far ? cap * t : z * p;
}

// tanh(x) / x for |x| <= 1 as a polynomial of y = x^2 (a Chebyshev fit of its relative
// error, 5e-9; in fp32 7e-8).
__device__ __forceinline__ float loss_tanh(int k) {
  constexpr float c[8] = {1.f,          -0.33333275f,  0.13332108f,   -0.053867836f,
                          0.021456175f, -0.0079049394f, 0.0022732385f, -0.00035080130f};
  return c[k];
}

}  // namespace lora
