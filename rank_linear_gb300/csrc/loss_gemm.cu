// loss_gemm.cu -- the two products of the large-vocabulary loss on the tensor
// cores (include/lora_loss.h; ch05 "Acceleration principles: Triton kernels and
// fused LoRA", §5.7).
//
// First:   Z = X W^T by tiles of 256 tokens x 512 words of the vocabulary, which
//          leave TMEM as E = exp2(u), u = log2(e) c(z) - ref (ref: the target's, so
//          that a row's largest is some 1 at least) in bf16, or not at all, and as
//          fp32 sums over 128 columns; and the target's own u.
// Second:  dX = scale (E W) by tiles of 256 tokens x 512 of the hidden size, the
//          vocabulary being the length of the products.
//
// Structure (as the layers' GEMMs): persistent CTA pairs, tcgen05.mma.cta_group::2
// with M = 256 and two N = 256 halves a K step that share one A tile; a four-stage
// TMA ring; warp 0 loads, one thread of warp 1 of the even CTA issues, eight warps
// drain.  A half of the accumulator is released as soon as it is in registers, so
// that the next tile's products run under the exponentials.  Per tile and SM the
// tensor cores take 1024 cycles a K block; the first product's drain makes 256
// exponentials a thread (4096 cycles of the SM's 16 a cycle): hidden from a hidden
// size of about 512 on.
#include <cuda_bf16.h>

#include <atomic>

#include "host.h"
#include "loss.cuh"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int BM = kLossTileM / 2, BK = kLossBlockK, BN = 256;  // rows of a CTA; K block; width of one MMA
constexpr int TN = kLossTileN;
constexpr int CLUSTER = 2;
constexpr uint16_t PAIR_MASK = 0x3;
constexpr uint32_t A_BYTES = BM * BK * 2, B_HALF = BN / 2 * BK * 2, B_BYTES = 2 * B_HALF;
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;  // 48 KB
constexpr int STAGES = 4;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t EPI_PITCH = 128, EPI_WARP_BYTES = 32 * EPI_PITCH;

struct __align__(16) Tail {
  uint64_t full[STAGES];   // even CTA: both CTAs' loads of a stage landed
  uint64_t empty[STAGES];  // each CTA: the pair's MMAs finished reading a stage
  uint64_t tfull;          // each CTA: the accumulator is complete
  uint64_t tempty[2];      // even CTA: both CTAs read a half out
  uint64_t drain;
  uint64_t peer_done;      // even CTA: the odd CTA's counts are in peer_issued
  uint64_t settled;        // odd CTA: the even CTA saw every copy of the pair land
  uint32_t tmem_base;
  int abort_flag;
  uint32_t peer_issued[STAGES];
};
constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + EPI_WARPS * EPI_WARP_BYTES + sizeof(Tail);
static_assert(SMEM <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Lane r's 64 numbers as row r of a staging chunk in the maps' 128-byte swizzle.
__device__ __forceinline__ void stage64(const float *v, uint8_t *stage, int lane) {
  uint4 *my = reinterpret_cast<uint4 *>(stage + lane * EPI_PITCH);
  const int sw = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    my[i ^ sw] = make_uint4(loss_pack(v[8 * i], v[8 * i + 1]), loss_pack(v[8 * i + 2], v[8 * i + 3]),
                            loss_pack(v[8 * i + 4], v[8 * i + 5]), loss_pack(v[8 * i + 6], v[8 * i + 7]));
}

// The first product's drain of 128 columns of a row (in v): sums, and
// exponentials in their place.  u = log2(e) c(z) - ref.  real: the row is a token's
// (else it is what the workspace held, which decides nothing for the others).  keep:
// takes the target's u where it is one of the columns.
template <bool CAP, class Keep>
__device__ __forceinline__ LossPart exponentials(float (&v)[kLossPiece], float ref, int target, bool real,
                                                 int col0, int n, float cap, float inv_cap, const Keep &keep) {
  constexpr float kLog2e = 1.4426950408889634f;
  // columns past the vocabulary, and the target's, which is added later: both are rare,
  // so that the whole warp looks once
  const bool mine = static_cast<unsigned>(target - col0) < unsigned(kLossPiece);
  const bool odd = col0 + kLossPiece > n || mine;
  const bool any_odd = __any_sync(0xffffffffu, odd);
  auto out = [&](int i) { return col0 + i >= n || col0 + i == target; };
  if constexpr (!CAP) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kLossPiece; ++i) {
      v[i] = fmaf(v[i], kLog2e, -ref);
      top = fmaxf(top, v[i]);
    }
    if (any_odd) {
      top = -INFINITY;
      float u = 0.f;
#pragma unroll
      for (int i = 0; i < kLossPiece; ++i) {
        if (col0 + i == target) u = v[i];
        if (out(i)) v[i] = -INFINITY;
        top = fmaxf(top, v[i]);
      }
      if (mine) keep(u);
    }
    LossPart p = {0.f, 0.f};
    if (top > kLossFar) {
      p.up = ceilf(top);
#pragma unroll
      for (int i = 0; i < kLossPiece; ++i) v[i] -= p.up;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kLossPiece; ++i) {
      v[i] = ex2(v[i]);
      s[i & 3] += v[i];
    }
    p.sum = (s[0] + s[1]) + (s[2] + s[3]);
    return p;
  } else {
    // what is kept is exp2(u) c'(z)
    if (any_odd) {
      float z = 0.f, slope;
#pragma unroll
      for (int i = 0; i < kLossPiece; ++i)
        if (col0 + i == target) z = v[i];
      if (mine) keep(fmaf(loss_cap(z, cap, inv_cap, slope), kLog2e, -ref));
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < kLossPiece; ++i) big = fmaxf(big, fabsf(v[i]));
    LossPart p = {0.f, 0.f};
    // Where no score of the warp is beyond the cap, nor any u far (|c(z)| <= |z|): a
    // polynomial, two scores an instruction.  (With the exponential form for all,
    // 2048 x 32000 x 4096 took 355 us where 294 without a cap: a half of the
    // accumulator waits for the other's exponentials.)
    if (__all_sync(0xffffffffu, !real || (big <= cap && fmaf(big, kLog2e, -ref) <= kLossFar))) {
      float2 s2 = make_float2(0.f, 0.f);
      const float2 inv2 = make_float2(inv_cap, inv_cap);
#pragma unroll
      for (int i = 0; i < kLossPiece; i += 2) {
        const float2 z = make_float2(v[i], v[i + 1]), x = __fmul2_rn(z, inv2), y = __fmul2_rn(x, x);
        float2 q = make_float2(loss_tanh(7), loss_tanh(7));
#pragma unroll
        for (int k = 6; k >= 0; --k) q = __ffma2_rn(q, y, make_float2(loss_tanh(k), loss_tanh(k)));
        const float2 t = __fmul2_rn(x, q);
        const float2 slope = __ffma2_rn(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f));
        const float2 u = __ffma2_rn(__fmul2_rn(z, q), make_float2(kLog2e, kLog2e), make_float2(-ref, -ref));
        float2 e = make_float2(ex2(u.x), ex2(u.y));
        if (any_odd) {
          if (out(i)) e.x = 0.f;
          if (out(i + 1)) e.y = 0.f;
        }
        s2 = __fadd2_rn(s2, e);
        e = __fmul2_rn(e, slope);
        v[i] = e.x;
        v[i + 1] = e.y;
      }
      p.sum = s2.x + s2.y;
      return p;
    }
    // c rises, so that the largest z decides
    if (any_odd) {
#pragma unroll
      for (int i = 0; i < kLossPiece; ++i)
        if (out(i)) v[i] = -INFINITY;
    }
    float top = -INFINITY, slope;
#pragma unroll
    for (int i = 0; i < kLossPiece; ++i) top = fmaxf(top, v[i]);
    top = fmaf(loss_cap(top, cap, inv_cap, slope), kLog2e, -ref);
    if (top > kLossFar) p.up = ceilf(top);
    const float off = ref + p.up;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kLossPiece; ++i) {
      float e = ex2(fmaf(loss_cap(v[i], cap, inv_cap, slope), kLog2e, -off));
      if (any_odd && out(i)) e = 0.f;
      s[i & 3] += e;
      v[i] = e * slope;
    }
    p.sum = (s[0] + s[1]) + (s[2] + s[3]);
    return p;
  }
}

// KIND 0: sums only, 1: sums and E, 2: dX.
template <int KIND, bool CAP>
__global__ void __launch_bounds__(THREADS, 1)
    k_loss_gemm(const __grid_constant__ LossGemm g) {
  constexpr bool GRAD = KIND == 2;  // B is MN-major: rows of W are the K index
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *epi_stage = smem_raw + (base - raw) + STAGES * STAGE_BYTES;
  auto *tail = reinterpret_cast<Tail *>(epi_stage + EPI_WARPS * EPI_WARP_BYTES);
  const uint32_t sA = base, sB = base + STAGES * A_BYTES;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int q = static_cast<int>(cluster_ctarank());
  const bool leader = q == 0;
  const int pair_id = blockIdx.x / CLUSTER, num_pairs = gridDim.x / CLUSTER;
  volatile int *abort_flag = &tail->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&tail->full[s]), 1);
      mbar_init(smem_u32(&tail->empty[s]), 1);
    }
    mbar_init(smem_u32(&tail->tfull), 1);
    for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&tail->tempty[h]), EPI_WARPS * CLUSTER);
    mbar_init(smem_u32(&tail->drain), 1);
    mbar_init(smem_u32(&tail->peer_done), 1);
    mbar_init(smem_u32(&tail->settled), 1);
    tail->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&g.a);
    tma_prefetch(&g.b);
    if (KIND == 1) tma_prefetch(&g.e);
  }
  cluster_sync();  // both CTAs' barriers exist before either signals the other's
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tail->tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  griddep_wait();  // the tokens that count, and what the kernels before wrote
  fence_proxy_async_global();  // ... for the copies that this thread issues
  griddep_launch_dependents();  // (the next kernel waits for this one's end itself)

  const int M = max(0, min(g.strip, g.head->live - g.first));
  const int m_pairs = (M + kLossTileM - 1) / kLossTileM, n_tiles = (g.n + TN - 1) / TN;
  const int kb_total = (g.k + BK - 1) / BK;
  const LossShare share = loss_share(m_pairs * n_tiles, num_pairs, kb_total);
  // item i of this pair; part: of the second product the slot of a range, of the
  // first the half of a tile (-1: none, it is a whole one)
  auto item = [&](int i, int &tile, int &lo, int &hi, int &part) -> bool {
    if constexpr (GRAD) return loss_item(share, pair_id, i, kb_total, tile, lo, hi, part);
    lo = 0;
    hi = kb_total;
    return loss_first_item(share.tiles, num_pairs, pair_id, i, tile, part);
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t issued[STAGES];
      for (int s = 0; s < STAGES; ++s) issued[s] = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int tile, lo, hi, part;
      uint32_t tx = STAGE_BYTES;  // what each CTA brings to a stage of the item
      for (int i = 0; ok && item(i, tile, lo, hi, part); ++i) {
        int mp, nb;
        loss_tile(tile, m_pairs, n_tiles, g.group, mp, nb);
        const bool narrow = !GRAD && part >= 0;  // half a tile: it takes the first half's place
        const int m0 = (2 * mp + q) * BM, n0 = nb * TN + q * (BN / 2) + (narrow ? part * BN : 0);
        if (narrow) tx = A_BYTES + B_HALF;
        for (int kb = lo; kb < hi; ++kb) {
          if (!mbar_wait(smem_u32(&tail->empty[stage]), phase ^ 1u, abort_flag, g.dev_status)) {
            ok = false;
            break;
          }
          const uint32_t full_local = smem_u32(&tail->full[stage]);
          const uint32_t full = dsmem_map(full_local, 0);
          if (leader) mbar_expect_tx(full_local, CLUSTER * tx);
          const int k0 = kb * BK;
          tma_load_2d_pair(sA + stage * A_BYTES, &g.a, full, k0, m0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && narrow) break;
            const uint32_t dst = sB + stage * B_BYTES + h * B_HALF;
            if constexpr (GRAD) {
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tma_load_2d_pair(dst + j * 8192u, &g.b, full, n0 + h * BN + 64 * j, k0);
            } else {
              tma_load_2d_pair(dst, &g.b, full, k0, n0 + h * BN);
            }
          }
          issued[stage] += 1;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      bool clean = ok;
      if (ok) {
        for (int s = 0; s < STAGES; ++s)
          if (issued[s] && !mbar_wait(smem_u32(&tail->empty[s]), (issued[s] - 1u) & 1u, abort_flag,
                                      g.dev_status)) {
            clean = false;
            break;
          }
      }
      // Both CTAs' copies complete on the even CTA's barriers.  The odd CTA
      // hands over how often it filled each stage and, when aborting, stays
      // until the even CTA, which settles the phases that only one of them
      // armed or filled (their counts differ by one at most; such a phase is one
      // of the item that the even CTA is at), has seen every copy land.
      if (!leader) {
        const uint32_t pi = smem_u32(tail->peer_issued);
        for (int s = 0; s < STAGES; ++s) dsmem_st_u32(dsmem_map(pi + 4u * s, 0), issued[s]);
        mbar_arrive_cluster(dsmem_map(smem_u32(&tail->peer_done), 0));
        if (!clean) mbar_wait_drain(smem_u32(&tail->settled), 0);
      } else {
        if (!clean) {
          const bool counts = mbar_wait_drain<true>(smem_u32(&tail->peer_done), 0);
          for (int s = 0; s < STAGES; ++s) {
            const uint32_t e = issued[s];
            const uint32_t o =
                counts ? reinterpret_cast<volatile uint32_t *>(tail->peer_issued)[s] : e;
            const uint32_t n = e > o ? e : o;
            if (n == 0) continue;
            const uint32_t fs = smem_u32(&tail->full[s]);
            if (e == o + 1)
              mbar_complete_tx(fs, tx);
            else if (o == e + 1)
              mbar_expect_tx(fs, tx);
            mbar_wait_drain(fs, (n - 1u) & 1u);
          }
        }
        mbar_arrive_cluster(dsmem_map(smem_u32(&tail->settled), 1));
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer (even CTA)
    if (leader && lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(CLUSTER * BM, BN, false, GRAD);
      constexpr uint64_t A_STEP = 32 >> 4, B_STEP = GRAD ? (2048 >> 4) : (32 >> 4);
      const uint64_t a0 = sdesc_sw128(sA, 16, 1024);
      const uint64_t b0 = GRAD ? sdesc_sw128(sB, 8192, 1024) : sdesc_sw128(sB, 16, 1024);
      auto issue = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t accum) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          tc_mma_bf16_pair(d, ad + kk * A_STEP, bd + kk * B_STEP, idesc, kk ? 1u : accum);
      };
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int tile, lo, hi, part;
      for (int i = 0; ok && item(i, tile, lo, hi, part); ++i) {
        const bool narrow = !GRAD && part >= 0;
        const uint32_t free = (static_cast<uint32_t>(i) & 1u) ^ 1u;
        if (!mbar_wait(smem_u32(&tail->tempty[0]), free, abort_flag, g.dev_status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        bool half1_free = false;
        uint64_t ad = a0 + stage * (A_BYTES >> 4), bd = b0 + stage * (B_BYTES >> 4);
        uint32_t accum = 0, accum1 = 0;
        // while the last tile's half 1 is still being read out, the half-0
        // products of up to STAGES - 1 blocks go ahead
        int deferred = 0;
        for (int kb = lo; kb < hi; ++kb) {
          if (!mbar_wait(smem_u32(&tail->full[stage]), phase, abort_flag, g.dev_status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue(tmem_base, ad, bd, accum);
          accum = 1u;
          bool hold = false;
          if (!narrow && !half1_free) {
            if (deferred + 1 < STAGES && kb + 1 < hi && !mbar_peek(smem_u32(&tail->tempty[1]), free)) {
              ++deferred;
              hold = true;
            } else {
              if (!mbar_wait(smem_u32(&tail->tempty[1]), free, abort_flag, g.dev_status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              half1_free = true;
              for (int j = deferred; j > 0; --j) {  // oldest first
                const int sj = stage >= j ? stage - j : stage - j + STAGES;
                issue(tmem_base + BN, a0 + sj * (A_BYTES >> 4),
                      b0 + sj * (B_BYTES >> 4) + (B_HALF >> 4), accum1);
                accum1 = 1u;
                tc_commit_pair_mc(smem_u32(&tail->empty[sj]), PAIR_MASK);
              }
              deferred = 0;
            }
          }
          if (!hold) {
            if (!narrow) issue(tmem_base + BN, ad, bd + (B_HALF >> 4), accum1);
            accum1 = 1u;
            tc_commit_pair_mc(smem_u32(&tail->empty[stage]), PAIR_MASK);
          }
          ad += A_BYTES >> 4;
          bd += B_BYTES >> 4;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
            ad = a0;
            bd = b0;
          }
        }
        if (!ok) break;
        tc_commit_pair_mc(smem_u32(&tail->tfull), PAIR_MASK);
      }
      if (!ok) {  // the products in flight end before TMEM is freed
        tc_commit_pair(smem_u32(&tail->drain));
        mbar_wait_drain(smem_u32(&tail->drain), 0);
      }
    }
  } else {
    // ------------------------------------------------------ drain (both CTAs)
    const int qd = warp & 3, cpart = (warp - 2) >> 2;  // lane quadrant; which 128 columns of a half
    uint8_t *stage = epi_stage + (warp - 2) * EPI_WARP_BYTES;
    const float inv_cap = CAP ? 1.f / g.cap : 0.f;
    int tile, lo, hi, part;
    for (int i = 0; item(i, tile, lo, hi, part); ++i) {
      int mp, nb;
      loss_tile(tile, m_pairs, n_tiles, g.group, mp, nb);
      const bool narrow = !GRAD && part >= 0;
      const int rl = qd * 32 + lane;  // row of this CTA's 128
      const int row0 = (2 * mp + q) * BM + qd * 32, row = row0 + lane;
      float ref = 0.f;  // first product: the row's reference; second: its factor
      int target = -1;
      if (row < M) {
        ref = GRAD ? g.scale[row] : g.ref[row];
        if (!GRAD) target = g.target[row];
      }
      const bool got = mbar_wait(smem_u32(&tail->tfull), static_cast<uint32_t>(i) & 1u, abort_flag,
                                 g.dev_status);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(qd * 32) << 16);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (narrow && h == 1) {  // (nothing there: the barrier's phases go on)
          if (lane == 0) mbar_arrive_cluster(dsmem_map(smem_u32(&tail->tempty[1]), 0));
          break;
        }
        // first column within the tile, and where it is in TMEM
        const int c0 = (narrow ? part : h) * BN + cpart * kLossPiece, at = h * BN + cpart * kLossPiece;
        float v[kLossPiece];
#pragma unroll
        for (int c = 0; c < kLossPiece / 32; ++c)
          tmem_ld_32cols(taddr + at + c * 32, *reinterpret_cast<float(*)[32]>(v + c * 32));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(dsmem_map(smem_u32(&tail->tempty[h]), 0));
        const int col0 = nb * TN + c0;
        if constexpr (!GRAD) {
          const LossPart p = exponentials<CAP>(v, ref, target, row < M, col0, g.n, g.cap, inv_cap,
                                               [&](float u) { g.own[row] = u; });
          g.parts[int64_t((nb * TN + c0) / kLossPiece) * g.strip + row] = p;
          if constexpr (KIND == 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // a box of 32 x 64 each, cut at the vocabulary's end
              if (lane == 0) bulk_wait_group_read0();
              __syncwarp();
              stage64(v + 64 * c, stage, lane);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0 && col0 + 64 * c < g.n && row0 < M) {
                tma_store_2d(&g.e, smem_u32(stage), col0 + 64 * c, row0);
                bulk_commit_group();
              }
            }
          }
        } else if (part >= 0) {
          // a range: the fp32 sums, column by column of 128 rows
          float *out = g.slots + size_t(part) * kLossSlotFloats + size_t(q) * (BM * TN) + rl;
#pragma unroll
          for (int c = 0; c < kLossPiece; ++c) out[(c0 + c) * BM] = v[c];
        } else {
          const int seg = lane & 7;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int k = 0; k < 64; ++k) v[64 * c + k] *= ref;
            stage64(v + 64 * c, stage, lane);
            __syncwarp();
            const int col = col0 + 64 * c + seg * 8;  // of this lane's 16 bytes
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // four rows an instruction, 128 bytes of each
              const int r = 4 * j + (lane >> 3);
              const uint4 o = *reinterpret_cast<const uint4 *>(stage + r * EPI_PITCH +
                                                               ((seg ^ (r & 7)) * 16));
              if (row0 + r < M && col < g.n)  // n is a multiple of 8
                *reinterpret_cast<uint4 *>(g.out + int64_t(g.place[row0 + r]) * g.ldo + col) = o;
            }
            __syncwarp();
          }
        }
      }
    }
    if (KIND == 1 && lane == 0) bulk_wait_group0();  // the stores are complete
  }

  __syncthreads();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int KIND, bool CAP>
cudaError_t launch(const LossGemm &g, int pairs, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  auto kern = &k_loss_gemm<KIND, CAP>;
  const cudaError_t e = allow_smem(kern, SMEM, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * CLUSTER));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CLUSTER;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, g);
}

}  // namespace

int loss_pairs(int num_sms) {
  const int n = main_gemm_pairs(true, num_sms);  // clusters of two with as much shared memory
  return n < kLossMaxPairs ? n : kLossMaxPairs;
}

cudaError_t launch_loss_gemm(int kind, const LossGemm &g, int pairs, cudaStream_t s) {
  if (kind == 2) return launch<2, false>(g, pairs, s);
  if (g.cap > 0.f) return kind == 1 ? launch<1, true>(g, pairs, s) : launch<0, true>(g, pairs, s);
  return kind == 1 ? launch<1, false>(g, pairs, s) : launch<0, false>(g, pairs, s);
}

}  // namespace lora
