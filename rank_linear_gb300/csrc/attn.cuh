// attn.cuh -- device code shared by the tensor-core attention kernels:
// 128 x 128 tiles of scores, which of them a mask leaves (wholly or partly),
// the transform of a score, and the tcgen05 forms with an operand in TMEM.
#pragma once

#include <cuda_bf16.h>

#include <climits>

#include "attn.h"
#include "ptx.cuh"

namespace lora {

constexpr int kTile = 128;  // rows of a query tile, and of a key tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- PTX forms
// The MMAs of a tile are issued by a whole warp with all but one lane
// predicated off: no divergent branch, so that descriptors stay in uniform
// registers.  (Under `if (lane == 0)` each issue took about 100 cycles, longer
// than the 64 of the MMA itself.)
//
// 1 in one lane of the warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
// A value that all lanes hold, as one the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }
// D(tmem) (+)= A(smem) * B(smem)^T.
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// D(tmem) (+)= A(tmem) * B(smem)^T: A is bf16, lane = row, two K elements per
// 32-bit column (16 K elements: 8 columns).
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of the warp's 32 lanes; the values are there after tmem_wait_ld
// and pin.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Keeps the uses of loaded registers after the wait before it.
template <int N>
__device__ __forceinline__ void pin(float *v) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]),
                      "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *v) {
  const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Tiled copies over [batch][head][token][dim] maps: x is the element of the head.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *tm, uint32_t bar,
                                            int32_t x, int32_t token, int32_t head, int32_t batch) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(token), "r"(head), "r"(batch)
      : "memory");
}
// The same over [batch][head / P][token][head modulo P][dim] maps, P heads of a
// token side by side.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *tm, uint32_t bar,
                                            int32_t x, int32_t token, int32_t heads, int32_t batch) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(0), "r"(token), "r"(heads),
      "r"(batch)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap *tm, int32_t x, int32_t token,
                                                int32_t head, int32_t batch) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(x), "r"(token), "r"(head), "r"(batch)
               : "memory");
}
// A warpgroup gives back registers above N, or waits for N to be free.
template <int N>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
        "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&p);
}

// A bounded wait of a whole warp: one answer for all lanes, and little code
// (the issuing warp's path from one product to the next is what the tensor
// core waits for).
__device__ __forceinline__ bool wait_warp(const uint64_t &bar, int phase, volatile int *abort_flag,
                                          unsigned *dev_status) {
  const uint32_t at = smem_u32(&bar);
  uint64_t t0 = 0;
  while (!__all_sync(~0u, mbar_test(at, phase & 1))) {
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    const bool late = now - t0 > kWaitLimitNs;
    if (__any_sync(~0u, late || *abort_flag != 0)) {
      if (threadIdx.x % 32 == 0 && *abort_flag == 0) {
        *abort_flag = 1;
        atomicOr(dev_status, kDevErrTimeout);
      }
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------- masks
// Documents of one 128-token tile: the range of those >= 0 (lo > hi: none),
// and whether some token is padding.
struct DocRange {
  int lo, hi, padded, unused;
};
__device__ __forceinline__ DocRange doc_range(const int4 *ranges, int64_t i) {
  const int4 r = __ldcg(ranges + i);
  return {r.x, r.y, r.z, r.w};
}
__device__ __forceinline__ bool docs_meet(const DocRange &a, const DocRange &b) {
  return a.lo <= b.hi && b.lo <= a.hi;  // an empty range has lo = INT_MAX, hi = -1
}
__device__ __forceinline__ bool docs_equal(const DocRange &a, const DocRange &b) {
  return a.lo == a.hi && b.lo == a.lo && b.hi == a.lo && !a.padded && !b.padded;
}

// By a whole warp, for a query tile of documents qr over the key tiles [0, hi):
// those from lo on that it may see (to the new hi), and of them those that
// share its one document, if they lie in one run: [same[0], same[1]).
__device__ __forceinline__ void doc_tiles(const DocRange &qr, const int4 *k_ranges, int &lo,
                                          int &hi, int (&same)[2]) {
  int from = INT_MAX, to = 0, first = INT_MAX, last = 0, equal = 0;
  for (int x = threadIdx.x % 32; x < hi; x += 32) {
    const DocRange kr = doc_range(k_ranges, x);
    if (docs_meet(qr, kr)) {
      from = min(from, x);
      to = x + 1;
    }
    if (docs_equal(qr, kr)) {
      first = min(first, x);
      last = x + 1;
      ++equal;
    }
  }
  hi = __reduce_max_sync(~0u, to);
  lo = min(__reduce_min_sync(~0u, from), hi);
  same[0] = __reduce_min_sync(~0u, first);
  same[1] = __reduce_max_sync(~0u, last);
  if (__reduce_add_sync(~0u, equal) != same[1] - same[0]) same[1] = same[0];
}

// Bits 0..n of a word (none for n < 0, all for n >= 31).
__device__ __forceinline__ uint32_t bits_to(int n) {
  return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1u;
}
// For each lane's own document, which of 32 W tokens share it: bit i of word c
// is token 32 c + i, whose document lane i holds in theirs[c] (below zero:
// padding).  A turn for every distinct document among the lanes.
template <int W>
__device__ __forceinline__ void same_doc(int own, const int (&theirs)[W], uint32_t (&keep)[W]) {
  uint32_t todo = __ballot_sync(~0u, own >= 0);
#pragma unroll
  for (int c = 0; c < W; ++c) keep[c] = 0u;
  while (todo != 0u) {
    const int doc = __shfl_sync(~0u, own, __ffs(todo) - 1);
    const bool mine = own == doc;
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const uint32_t b = __ballot_sync(~0u, theirs[c] == doc);
      if (mine) keep[c] = b;
    }
    todo &= ~__ballot_sync(~0u, mine);
  }
}
// Documents of 32 W tokens from docs on, `have` of them there.
template <int W>
__device__ __forceinline__ void load_docs(const int *docs, int have, int (&out)[W]) {
#pragma unroll
  for (int c = 0; c < W; ++c) {
    const int i = 32 * c + static_cast<int>(threadIdx.x % 32);
    out[c] = i < have ? docs[i] : -1;
  }
}

// What a query of position p (its row's index + Sk - Sq) sees without
// documents: the keys up to this one (below 0: none).
__device__ __forceinline__ int last_key(const AttnArgs &a, int p, int prefix) {
  const int lim = a.causal ? max(p, prefix - 1) : a.Sk - 1;
  return min(lim, a.Sk - 1);
}

// The score of a raw product z = q . k, in units of log 2, without the mask.
// CAP: c = cap tanh x, x = z scale / cap, by one of two ways for all of a
// warp's pairs at hand:
//  - |x| <= 1 for all of them: x P(x^2), P the polynomial of degree 5 next to tanh(x) / x on
//    [0, 1] (a reweighted least-squares fit; the error of tanh is 2.4e-7 at the
//    most, 3.1e-6 of itself next to 0), two pairs an instruction;
//  - else tanh x = 1 - 2 r, r = 1 / (1 + e^2x): two more special functions a
//    pair, of which an SM does 32 a cycle.  Its absolute error is 2^-22 of the
//    cap, which would drown scores far below a large cap: for |x| <= 1/8 the
//    series' first terms, x - x^3 / 3 + 2 x^5 / 15 (2e-7 of it is left out).
// What x is formed from is bounded, so that no cap, however small or large,
// makes 0 times infinity of a product that is 0 (as rows past the end are) or
// of its tanh.
__device__ __forceinline__ constexpr float tanh_poly(int i) {  // P's coefficients
  return i == 0 ? 0.99999685f : i == 1 ? -0.33324004f : i == 2 ? 0.13253524f : i == 3 ? -0.050972835f
         : i == 4 ? 0.016114152f : -0.0028394550f;
}
struct ScoreConst {
  float scale2;    // scale * log2 e
  float x_by;      // scale / cap
  float cap2;      // cap * log2 e
  float slope2;    // slope * log2 e
  float most;      // cap / scale: the largest |z| for the polynomial
  float top;       // what tanh is multiplied by at once: cap2, or 1
  float poly[6];   // P times that
};
__device__ __forceinline__ ScoreConst score_const(const AttnArgs &a, int head, bool unit = false) {
  constexpr float kBig = 3e38f;
  ScoreConst c;
  c.scale2 = a.scale * kLog2e;
  c.slope2 = a.slopes != nullptr ? a.slopes[head] * kLog2e : 0.f;
  c.x_by = c.cap2 = c.most = c.top = 0.f;
  if (a.cap > 0.f) {
    c.x_by = fminf(a.scale / a.cap, kBig / 4.f);  // (its e^2x takes 2 log2 e of it)
    c.cap2 = fminf(a.cap * kLog2e, kBig / 2.f);   // (1 - 2 r takes 2 of it)
    c.most = fminf(a.cap / a.scale, kBig);        // infinite products are beyond it
    c.top = unit ? 1.f : c.cap2;
#pragma unroll
    for (int i = 0; i < 6; ++i) c.poly[i] = tanh_poly(i) * c.top;
  }
  return c;
}
// Are the N products of every lane the polynomial's?
template <int N>
__device__ __forceinline__ bool all_small(const ScoreConst &c, const float *z) {
  float m[2] = {fabsf(z[0]), fabsf(z[1])};
#pragma unroll
  for (int j = 2; j + 2 < N; j += 4)
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = max3(m[i], fabsf(z[j + 2 * i]), fabsf(z[j + 2 * i + 1]));
  m[0] = max3(m[0], fabsf(z[N - 2]), fabsf(z[N - 1]));
  return __all_sync(~0u, fmaxf(m[0], m[1]) <= c.most);
}
// top tanh x of two pairs that are.
__device__ __forceinline__ float2 cap_small(const ScoreConst &c, float2 z) {
  const float2 x = mul2(z, make_float2(c.x_by, c.x_by)), u = mul2(x, x);
  float2 p = make_float2(c.poly[5], c.poly[5]);
#pragma unroll
  for (int i = 4; i >= 0; --i) p = fma2(p, u, make_float2(c.poly[i], c.poly[i]));
  return mul2(x, p);
}
// The same by the series, good for |x| <= 1/8.
__device__ __forceinline__ float2 cap_near(const ScoreConst &c, float2 z) {
  const float2 x = mul2(z, make_float2(c.x_by, c.x_by)), u = mul2(x, x);
  const float2 y = mul2(x, make_float2(c.top, c.top));
  const float2 p = fma2(u, make_float2(2.f / 15.f, 2.f / 15.f), make_float2(-1.f / 3.f, -1.f / 3.f));
  return fma2(mul2(u, p), y, y);
}
// r as above of z, or of |z|: dc/dz = scale * 4 r (1 - r), which is good where
// |tanh| is next to 1 with the r of |z| only.
__device__ __forceinline__ float cap_r(const ScoreConst &c, float z) {
  return rcp(1.f + ex2(z * (2.f * kLog2e * c.x_by)));
}
// top tanh x of any pair from its r; near: from the series.
__device__ __forceinline__ float cap_any(const ScoreConst &c, float z, float r, float near) {
  return fabsf(z) <= 0.125f * c.most ? near : fmaf(-2.f * c.top, r, c.top);
}
// Two scores; small: what all_small said of them.
template <bool CAP, bool BIAS>
__device__ __forceinline__ float2 scores2(const ScoreConst &c, float2 z, float distance, float step,
                                          bool small) {
  float2 s;
  if constexpr (CAP) {
    if (small) {
      s = cap_small(c, z);
    } else {
      s = cap_near(c, z);
      s = make_float2(cap_any(c, z.x, cap_r(c, z.x), s.x), cap_any(c, z.y, cap_r(c, z.y), s.y));
    }
  } else {
    s = mul2(z, make_float2(c.scale2, c.scale2));
  }
  if constexpr (BIAS) {
    s.x = fmaf(-c.slope2, fabsf(distance), s.x);
    s.y = fmaf(-c.slope2, fabsf(distance + step), s.y);
  }
  return s;
}

// Zeroes the rows of a [128][DH] tile (64-wide boxes of 128-byte rows) whose
// token is padding, by one warp, so that an operand's rows that no score
// uses cannot turn a zero weight into NaN.  docs: the tile's first token.
template <int DH>
__device__ __forceinline__ void zero_padding_rows(uint8_t *tile, const int *docs, int rows) {
  for (int r = threadIdx.x % 32; r < kTile; r += 32)
    if (r < rows && docs[r] < 0)
      for (int box = 0; box < DH / 64; ++box)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4 *>(tile + box * kTile * 128 + r * 128 + i * 16) =
              make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// Stores 32 columns from c on of the warp's 32 rows, row0 + lane being this
// lane's, as bf16 times the lane's factor: rows of D elements, `stride` apart,
// those from `end` on left out.  Four lanes first exchange 16-byte pieces so
// that a store writes 64 bytes of a row side by side: straight from the row
// owners it takes a request for every 16 bytes (2500 against 900 cycles for a
// tile of dq).  shift > 0: the rows are 2^shift heads, `head_stride` apart, of
// one token after the other.
__device__ __forceinline__ void store_rows32(__nv_bfloat16 *base, int64_t stride, int row0, int end,
                                             int c, int D, const float *v, float by, int shift = 0,
                                             int64_t head_stride = 0) {
  const int lane = threadIdx.x % 32;
  uint32_t w[4][4];  // pieces of this lane's row
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[i][e] = pack_bf16(v[i * 8 + 2 * e] * by, v[i * 8 + 2 * e + 1] * by);
  // the 4 x 4 pieces of four lanes transposed
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t got = __shfl_xor_sync(~0u, odd ? w[i][e] : w[i + 1][e], 1);
      if (odd)
        w[i][e] = got;
      else
        w[i + 1][e] = got;
    }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t got = __shfl_xor_sync(~0u, high ? w[i][e] : w[i + 2][e], 2);
      if (high)
        w[i][e] = got;
      else
        w[i + 2][e] = got;
    }
  // now w[i] is piece lane % 4 of row i of the four
  const int col = c + 8 * (lane & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + (lane & ~3) + i;
    if (row < end && col < D)
      *reinterpret_cast<uint4 *>(base + (row >> shift) * stride +
                                 (row & ((1 << shift) - 1)) * head_stride + col) =
          make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
}

// Operand descriptors of a [128][DH] tile as TMA leaves it (128-byte swizzle,
// boxes of 64 columns): with the head as K (K-major), or the tokens
// (MN-major); and what K step kk of 16 adds to each.
__device__ __forceinline__ uint64_t desc_head(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ constexpr uint64_t head_step(int kk) {
  return ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
}
__device__ __forceinline__ uint64_t desc_token(uint32_t tile) {
  return sdesc_sw128(tile, kTile * 128, 1024);
}
__device__ __forceinline__ constexpr uint64_t token_step(int kk) { return (kk * 2048) >> 4; }

// D = X Y^T over the head, X and Y [128][DH] tiles.
template <int DH>
__device__ __forceinline__ void mma_over_head(uint32_t on, uint32_t d_tmem, uint32_t x, uint32_t y) {
  const uint64_t xd = desc_head(x), yd = desc_head(y);
#pragma unroll
  for (int kk = 0; kk < DH / 16; ++kk)
    mma_ss(on, d_tmem, xd + head_step(kk), yd + head_step(kk),
           idesc_bf16(kTile, kTile, false, false), kk > 0);
}
// D (+)= W Y over the tokens of K steps [FROM, TO) of a tile, W the TMEM
// operand whose K step kk is at column cols(kk), Y a [128][DH] tile.
template <int DH, int FROM, int TO, class F>
__device__ __forceinline__ void mma_over_tokens(uint32_t on, uint32_t d_tmem, uint32_t w_tmem, F cols,
                                                uint32_t y, bool accumulate) {
  const uint64_t yd = desc_token(y);
#pragma unroll
  for (int kk = FROM; kk < TO; ++kk)
    mma_ts(on, d_tmem, w_tmem + cols(kk), yd + token_step(kk), idesc_bf16(kTile, DH, false, true),
           accumulate || kk > FROM);
}

}  // namespace lora
