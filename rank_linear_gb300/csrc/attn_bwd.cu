// attn_bwd.cu -- attention backward on the tensor cores (include/lora_attention.h).
//
// Two kernels, so that every sum has one owner and a fixed order (no atomics):
// one passes over the keys for 128 queries and keeps dq in TMEM, the other
// over the queries of all heads of a group for 128 keys and keeps dk and dv.
// Each recomputes the scores, seven products of 128 x 128 tiles in all where
// sharing them across blocks would take five.  What a thread computes for a
// pair, dz = P dc/dz (dP - delta) with P = exp(s - lse), goes back into TMEM
// as bf16 over the scores (or over dP) and is the TMEM operand of the products
// that follow; nothing of size q_len x k_len leaves the SM.
#include "attn.cuh"
#include "host.h"

namespace lora {
namespace {

// Two warpgroups for the pairs (128 rows, 64 columns each) and one of which
// two warps issue the copies and the MMAs; registers as in the forward.
constexpr int kThreads = 384, kPairThreads = 256, kPairRegs = 224, kIssueRegs = 56;

struct Params {
  AttnArgs a;
  AttnBwdMaps m;
};

// The columns of a 128-wide TMEM region that hold K step kk of a bf16 operand:
// the warpgroup of columns 0..63 writes columns 0..31, the other 64..95, each
// over scores that it alone reads.
__device__ __forceinline__ constexpr uint32_t operand_cols(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

// P (to p) and P dc/dz (in s) of 64 raw products of one thread; distances
// d0 + step * j; sub = -lse in log2 units (or one per column in sub_col).
template <bool CAP, bool BIAS, bool PER_COLUMN>
__device__ __forceinline__ void weights(const ScoreConst &c, float (&s)[64], float *p, float sub,
                                        const float *sub_col, float d0, float step) {
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    float4 sc;
    if constexpr (PER_COLUMN)
      sc = *reinterpret_cast<const float4 *>(sub_col + j);
    else
      sc = make_float4(sub, sub, sub, sub);
    const float add[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float2 x = make_float2(s[j + i], s[j + i + 1]);
      const float2 y = make_float2(add[i], add[i + 1]);
      float r0 = 0.f, r1 = 0.f;
      if constexpr (CAP || BIAS) {
        x.x = score2<CAP, BIAS>(c, x.x, d0 + step * (j + i), r0);
        x.y = score2<CAP, BIAS>(c, x.y, d0 + step * (j + i + 1), r1);
        x = add2(x, y);
      } else {
        x = fma2(x, make_float2(c.scale2, c.scale2), y);
      }
      x.x = ex2(x.x);
      x.y = ex2(x.y);
      if (p != nullptr) {
        p[j + i] = x.x;
        p[j + i + 1] = x.y;
      }
      if constexpr (CAP) {  // dc/dz = 1 - tanh^2 = 4 r (1 - r)
        x.x *= 4.f * r0 * (1.f - r0);
        x.y *= 4.f * r1 * (1.f - r1);
      }
      s[j + i] = x.x;
      s[j + i + 1] = x.y;
    }
  }
}

// ---------------------------------------------------------------- dq
// Shared memory: Q, dO, then rings of K and V tiles.  TMEM: the scores (then
// dz) of two tiles at 0 and 128, dP at 256, dq at 384.
template <int DH>
struct DqLayout {
  static constexpr uint32_t kTileBytes = kTile * DH * 2;
  static constexpr int kKSlots = 3, kVSlots = 2;
  static constexpr uint32_t kBytes = (2 + kKSlots + kVSlots) * kTileBytes;
  // one block per SM (TMEM): more than half of its shared memory
  static constexpr uint32_t kAsked = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
struct DqTail {
  uint64_t q_full, k_full[3], k_empty[3], v_full[2];
  uint64_t s_full[2], dp_full[2], dp_free, dz_full, done, drain;
  uint32_t tmem;
  int abort_flag, lo, hi;
  float delta[2][kTile];
};

template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) k_attn_dq(const __grid_constant__ Params p) {
  using L = DqLayout<DH>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  DqTail *tail = reinterpret_cast<DqTail *>(smem + L::kBytes);
  const AttnArgs &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  const int heads = a.B * a.Hq;
  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int qt = qtiles - 1 - static_cast<int>(blockIdx.x / heads);
  const int bh = blockIdx.x % heads, b = bh / a.Hq, h = bh % a.Hq, g = h / a.group;
  const int row0 = qt * kTile, off = a.Sk - a.Sq;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->q_full), 1);
    for (int s = 0; s < L::kKSlots; ++s) {
      mbar_init(smem_u32(&tail->k_full[s]), 1);
      mbar_init(smem_u32(&tail->k_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&tail->v_full[s]), 1);
      mbar_init(smem_u32(&tail->s_full[s]), 1);
      mbar_init(smem_u32(&tail->dp_full[s]), 1);
    }
    mbar_init(smem_u32(&tail->dp_free), kPairThreads);
    mbar_init(smem_u32(&tail->dz_full), kPairThreads);
    mbar_init(smem_u32(&tail->done), 1);
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    tail->lo = a.q_docs != nullptr ? INT_MAX : 0;
    tail->hi = 0;
    fence_barrier_init();
    tma_prefetch(&p.m.q);
    tma_prefetch(&p.m.k);
    tma_prefetch(&p.m.v);
    tma_prefetch(&p.m.d_o);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 9) {
    tmem_alloc(smem_u32(&tail->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tail->tmem);

  // ---- the key tiles that some row sees
  const int prefix = a.prefix != nullptr ? a.prefix[b] : 0;
  const int most =
      max(0, (last_key(a, min(row0 + kTile, a.Sq) - 1 + off, prefix) + kTile) / kTile);
  DocRange qr = {0, 0, 0, 0};
  if (a.q_docs != nullptr) {
    qr = doc_range(a.q_ranges, int64_t(b) * qtiles + qt);
    for (int n = threadIdx.x; n < most; n += kThreads)
      if (docs_meet(qr, doc_range(a.k_ranges, int64_t(b) * ktiles + n))) {
        atomicMin(&tail->lo, n);
        atomicMax(&tail->hi, n + 1);
      }
  } else if (threadIdx.x == 0) {
    tail->hi = most;
  }
  __syncthreads();
  const int end = uniform(tail->hi), begin = uniform(min(tail->lo, end));
  const int count = end - begin;

  if (warp >= 8) {
    set_max_regs_down<kIssueRegs>();
    const uint32_t q_tile = smem_u32(smem), do_tile = q_tile + L::kTileBytes;
    const uint32_t k_ring = do_tile + L::kTileBytes, v_ring = k_ring + L::kKSlots * L::kTileBytes;
    if (warp == 8) {
      // ------------------------------------------------------ TMA
      if (lane == 0 && count > 0) {
        auto load = [&](uint32_t dst, const CUtensorMap *tm, uint64_t &bar, int token, int head) {
          for (int c = 0; c < DH / 64; ++c)
            tma_load_4d(dst + c * kTile * 128, tm, smem_u32(&bar), c * 64, token, head, b);
        };
        mbar_expect_tx(smem_u32(&tail->q_full), 2 * L::kTileBytes);
        load(q_tile, &p.m.q, tail->q_full, row0, h);
        load(do_tile, &p.m.d_o, tail->q_full, row0, h);
        int nk = 0, nv = 0;
        for (int i = 0; i < count; ++i) {
          const int ks = i % L::kKSlots, vs = i % L::kVSlots;
          if (i >= L::kKSlots && !mbar_wait(smem_u32(&tail->k_empty[ks]), (i / L::kKSlots - 1) & 1,
                                            abort_flag, a.dev_status))
            break;
          mbar_expect_tx(smem_u32(&tail->k_full[ks]), L::kTileBytes);
          load(k_ring + ks * L::kTileBytes, &p.m.k, tail->k_full[ks], (begin + i) * kTile, g);
          ++nk;
          // dP of the tile before in this slot is done
          if (i >= L::kVSlots && !mbar_wait(smem_u32(&tail->dp_full[vs]), (i / L::kVSlots - 1) & 1,
                                            abort_flag, a.dev_status))
            break;
          mbar_expect_tx(smem_u32(&tail->v_full[vs]), L::kTileBytes);
          load(v_ring + vs * L::kTileBytes, &p.m.v, tail->v_full[vs], (begin + i) * kTile, g);
          ++nv;
        }
        // copies in flight land before the CTA leaves
        mbar_wait_drain(smem_u32(&tail->q_full), 0);
        for (int s = 0; s < L::kKSlots && s < nk; ++s)
          mbar_wait_drain(smem_u32(&tail->k_full[s]), ((nk - 1 - s) / L::kKSlots) & 1);
        for (int s = 0; s < L::kVSlots && s < nv; ++s)
          mbar_wait_drain(smem_u32(&tail->v_full[s]), ((nv - 1 - s) / L::kVSlots) & 1);
      }
    } else if (warp == 9 && count > 0) {
      // ------------------------------------------------------ MMA
      const uint32_t on = elect_one();
      auto wait = [&](const uint64_t &bar, int phase) {  // one answer for the warp
        return wait_warp(bar, phase, abort_flag, a.dev_status);
      };
      auto padded = [&](int i) {
        return a.q_docs != nullptr && i < count &&
               doc_range(a.k_ranges, int64_t(b) * ktiles + begin + i).padded;
      };
      // K's tile i has landed, without the rows of padding
      bool pads = padded(0);
      auto wait_k = [&](int i) {
        const int s = i % L::kKSlots;
        if (!wait(tail->k_full[s], i / L::kKSlots)) return false;
        const bool now = pads;
        pads = padded(i + 1);
        if (now)
          zero_padding_rows<DH>(smem + (2 + s) * L::kTileBytes,
                                a.k_docs + b * a.kds + (begin + i) * kTile,
                                a.Sk - (begin + i) * kTile);
        return true;
      };
      auto scores = [&](int i) {
        mma_over_head<DH>(on, tmem + (i & 1) * kTile, q_tile,
                          k_ring + (i % L::kKSlots) * L::kTileBytes);
        commit(on, smem_u32(&tail->s_full[i & 1]));
      };
      auto do_v = [&](int i) {
        mma_over_head<DH>(on, tmem + 256, do_tile, v_ring + (i % L::kVSlots) * L::kTileBytes);
        commit(on, smem_u32(&tail->dp_full[i % L::kVSlots]));
      };
      bool ok = wait(tail->q_full, 0) && wait_k(0);
      tc_fence_after();
      if (ok) scores(0);
      if (ok) ok = wait(tail->v_full[0], 0);
      tc_fence_after();
      if (ok) do_v(0);
      for (int i = 0; i < count && ok; ++i) {
        if (i + 1 < count) {
          // over the dz of tile i - 1, which its product (issued) reads first
          if (!(ok = wait_k(i + 1))) break;
          tc_fence_after();
          scores(i + 1);
          if (!(ok = wait(tail->v_full[(i + 1) % L::kVSlots], (i + 1) / L::kVSlots) &&
                     wait(tail->dp_free, i)))
            break;
          tc_fence_after();
          do_v(i + 1);
        }
        if (!(ok = wait(tail->dz_full, i))) break;
        tc_fence_after();
        mma_over_tokens<DH, 0, 8>(on, tmem + 384, tmem + (i & 1) * kTile, operand_cols,
                            k_ring + (i % L::kKSlots) * L::kTileBytes, i > 0);
        commit(on, smem_u32(&tail->k_empty[i % L::kKSlots]));
        __syncwarp();
      }
      if (ok) commit(on, smem_u32(&tail->done));
      commit(on, smem_u32(&tail->drain));
      mbar_wait_drain(smem_u32(&tail->drain), 0);
      __syncwarp();
    }
  } else {
    set_max_regs_up<kPairRegs>();
    // ------------------------------------------------------ pairs
    const int half = warp / 4, r = threadIdx.x & 127, row = row0 + r;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const ScoreConst sc = score_const(a, h);
    const int pos = row + off;
    const int last = row < a.Sq ? last_key(a, pos, prefix) : -1;
    const int first_last = last_key(a, row0 + off, prefix);
    const int64_t stat = (static_cast<int64_t>(b) * a.Hq + h) * a.Sq + row;
    const int qd = a.q_docs != nullptr && row < a.Sq ? a.q_docs[b * a.qds + row] : -1;
    // delta = do . o, half of the head in each warpgroup
    float delta = 0.f, sub = -INFINITY;
    if (row < a.Sq) {
      const __nv_bfloat16 *o = static_cast<const __nv_bfloat16 *>(a.o) + b * a.so[0] +
                               row * a.so[1] + h * a.so[2];
      const __nv_bfloat16 *e = static_cast<const __nv_bfloat16 *>(a.d_o) + b * a.sdo[0] +
                               row * a.sdo[1] + h * a.sdo[2];
#pragma unroll 4
      for (int c = half * 8; c < a.D; c += 16) {
        const uint4 x = *reinterpret_cast<const uint4 *>(o + c);
        const uint4 y = *reinterpret_cast<const uint4 *>(e + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          delta = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), delta);
          delta = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u),
                       delta);
        }
      }
      const float lse = a.lse[stat];
      sub = lse == -INFINITY ? -INFINITY : -lse * kLog2e;  // a row that sees nothing: P = 0
    }
    tail->delta[half][r] = delta;
    named_bar_sync(1, kPairThreads);
    delta = tail->delta[0][r] + tail->delta[1][r];
    if (half == 0 && row < a.Sq) a.delta[stat] = delta;
    bool ok = true;
    DocRange kr = {0, 0, 0, 0};
    if (a.q_docs != nullptr && count > 0) kr = doc_range(a.k_ranges, int64_t(b) * ktiles + begin);
    for (int i = 0; i < count; ++i) {
      const int n = begin + i, key0 = n * kTile + half * 64;
      bool whole = n * kTile + kTile - 1 <= first_last;
      int kd[2];
      if (a.q_docs != nullptr) {
        whole = whole && docs_equal(qr, kr);
        if (!whole) load_docs(a.k_docs + b * a.kds + key0, a.Sk - key0, kd);
        if (i + 1 < count) kr = doc_range(a.k_ranges, int64_t(b) * ktiles + n + 1);
      }
      const uint32_t s_addr = tmem + lanes + (i & 1) * kTile + half * 64;
      if (!(ok = wait_warp(tail->s_full[i & 1], i >> 1, abort_flag, a.dev_status))) break;
      tc_fence_after();
      float w[64];
      tmem_ld32(s_addr, w);
      tmem_ld32(s_addr + 32, w + 32);
      tmem_wait_ld();
      pin<64>(w);
      weights<CAP, BIAS, false>(sc, w, nullptr, sub, nullptr, static_cast<float>(pos - key0), -1.f);
      if (!whole) {
        uint32_t keep[2] = {~0u, ~0u};
        if (a.q_docs != nullptr) same_doc(qd, kd, keep);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          keep[c] &= bits_to(last - key0 - 32 * c);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(keep[c] >> j & 1u)) w[c * 32 + j] = 0.f;
        }
      }
      if (!(ok = wait_warp(tail->dp_full[i & 1], i >> 1, abort_flag, a.dev_status))) break;
      tc_fence_after();
      float dp[64];
      tmem_ld32(tmem + lanes + 256 + half * 64, dp);
      tmem_ld32(tmem + lanes + 256 + half * 64 + 32, dp + 32);
      tmem_wait_ld();
      pin<64>(dp);
      tc_fence_before();
      mbar_arrive(smem_u32(&tail->dp_free));
      const float2 nd = make_float2(-delta, -delta);
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        const float2 x = mul2(make_float2(w[j], w[j + 1]),
                              add2(make_float2(dp[j], dp[j + 1]), nd));
        dp[j] = x.x;
        dp[j + 1] = x.y;
      }
      if (!whole) {  // a masked pair's dP may be anything
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (w[j] == 0.f) dp[j] = 0.f;
      }
      uint32_t z[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) z[j] = pack_bf16(dp[2 * j], dp[2 * j + 1]);
      tmem_st16(s_addr, z);
      tmem_st16(s_addr + 16, z + 16);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&tail->dz_full));
    }
    if (ok && count > 0) {
      ok = wait_warp(tail->done, 0, abort_flag, a.dev_status);
    }
    if (ok) {  // dq through Q's shared memory, half of the columns each
      tc_fence_after();
#pragma unroll 1
      for (int c = half * (DH / 2); c < (half + 1) * (DH / 2); c += 32) {
        float o[32];
        if (count > 0) {
          tmem_ld32(tmem + lanes + 384 + c, o);
          tmem_wait_ld();
          pin<32>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        stage_row32(smem, r, c, o, a.scale);
      }
      fence_proxy_async_smem();
    }
    const bool failed = named_bar_red_or(1, kPairThreads, !ok);
    if (!failed && threadIdx.x == 0) {
      for (int c = 0; c < DH / 64; ++c)
        if (c * 64 < a.D)
          tma_store_4d(&p.m.dq, smem_u32(smem) + c * kTile * 128, c * 64, row0, h, b);
      bulk_commit_group();
      bulk_wait_group0();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dk, dv
// Shared memory: K, V, then rings of Q and dO tiles.  TMEM: the transposed
// scores (then P^T) at 0, dP^T (then dz^T) at 128, dv at 256, dk at 384.
template <int DH>
struct DkvLayout {
  static constexpr uint32_t kTileBytes = kTile * DH * 2;
  // Q is asked for half a step before dO
  static constexpr int kQSlots = 3, kESlots = 2;
  // the tiles follow the tail (DkvTail), which for a head of 128 fills what
  // they leave of an SM's 227 KB: no room to align a base that is not aligned
  static constexpr uint32_t kTailBytes = 3072;
  static constexpr uint32_t kBytes = kTailBytes + (2 + kQSlots + kESlots) * kTileBytes;
  static constexpr uint32_t kAsked = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
struct DkvTail {
  // per tile of queries: -lse in log2 units, and -delta
  float sub[2][kTile], neg_delta[2][kTile];
  uint64_t k_full, q_full[3], e_full[2];
  uint64_t s_full, dp_full, p_full, dz_full, done, drain;
  uint32_t tmem;
  int abort_flag, lo, hi;
};

template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) k_attn_dkv(const __grid_constant__ Params p) {
  using L = DkvLayout<DH>;
  extern __shared__ __align__(1024) uint8_t raw_dkv[];
  uint8_t *smem = raw_dkv + L::kTailBytes;
  DkvTail *tail = reinterpret_cast<DkvTail *>(raw_dkv);
  static_assert(sizeof(DkvTail) <= L::kTailBytes, "tail");
  const AttnArgs &a = p.a;
  if ((smem_u32(raw_dkv) & 1023) != 0) {  // not met: the tiles' layout needs it
    if (threadIdx.x == 0) atomicOr(a.dev_status, kDevErrTimeout);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  // the first keys of a causal mask are seen by most queries: first
  const int heads = a.B * a.Hk;
  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int kt = blockIdx.x / heads;
  const int bg = blockIdx.x % heads, b = bg / a.Hk, g = bg % a.Hk;
  const int key0 = kt * kTile, off = a.Sk - a.Sq;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->k_full), 1);
    for (int s = 0; s < L::kQSlots; ++s) mbar_init(smem_u32(&tail->q_full[s]), 1);
    for (int s = 0; s < L::kESlots; ++s) mbar_init(smem_u32(&tail->e_full[s]), 1);
    mbar_init(smem_u32(&tail->s_full), 1);
    mbar_init(smem_u32(&tail->dp_full), 1);
    mbar_init(smem_u32(&tail->p_full), kPairThreads);
    mbar_init(smem_u32(&tail->dz_full), kPairThreads);
    mbar_init(smem_u32(&tail->done), 1);
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    tail->lo = INT_MAX;
    tail->hi = 0;
    fence_barrier_init();
    tma_prefetch(&p.m.q);
    tma_prefetch(&p.m.k);
    tma_prefetch(&p.m.v);
    tma_prefetch(&p.m.d_o);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 9) {
    tmem_alloc(smem_u32(&tail->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tail->tmem);

  // ---- the query tiles that see some key
  const int prefix = a.prefix != nullptr ? a.prefix[b] : 0;
  const int first = a.causal && key0 >= prefix ? max(0, key0 - off) / kTile : 0;
  DocRange kr = {0, 0, 0, 0};
  if (a.q_docs != nullptr) {
    kr = doc_range(a.k_ranges, int64_t(b) * ktiles + kt);
    for (int n = first + threadIdx.x; n < qtiles; n += kThreads)
      if (docs_meet(kr, doc_range(a.q_ranges, int64_t(b) * qtiles + n))) {
        atomicMin(&tail->lo, n);
        atomicMax(&tail->hi, n + 1);
      }
  } else if (threadIdx.x == 0) {
    tail->lo = first;
    tail->hi = qtiles;
  }
  __syncthreads();
  const int end = uniform(tail->hi), begin = uniform(min(tail->lo, end));
  const int per_head = end - begin, count = per_head * a.group;
  // step i: query head g * group + i / per_head, tile begin + i % per_head

  if (warp >= 8) {
    set_max_regs_down<kIssueRegs>();
    const uint32_t k_tile = smem_u32(smem), v_tile = k_tile + L::kTileBytes;
    const uint32_t q_ring = v_tile + L::kTileBytes, e_ring = q_ring + L::kQSlots * L::kTileBytes;
    if (warp == 8) {
      // ------------------------------------------------------ TMA
      if (lane == 0 && count > 0) {
        auto load = [&](uint32_t dst, const CUtensorMap *tm, uint64_t &bar, int token, int head) {
          for (int c = 0; c < DH / 64; ++c)
            tma_load_4d(dst + c * kTile * 128, tm, smem_u32(&bar), c * 64, token, head, b);
        };
        mbar_expect_tx(smem_u32(&tail->k_full), 2 * L::kTileBytes);
        load(k_tile, &p.m.k, tail->k_full, key0, g);
        load(v_tile, &p.m.v, tail->k_full, key0, g);
        int nq = 0, ne = 0;
        auto load_q = [&](int i) {
          const int s = i % L::kQSlots;
          mbar_expect_tx(smem_u32(&tail->q_full[s]), L::kTileBytes);
          load(q_ring + s * L::kTileBytes, &p.m.q, tail->q_full[s],
               (begin + i % per_head) * kTile, g * a.group + i / per_head);
          ++nq;
        };
        load_q(0);
        for (int i = 0; i < count; ++i) {
          // dP of step i - 1 is done, hence everything of step i - 2: the slots
          // of Q's tile i - 2 and dO's
          // (every phase in turn: a wait for phase 1 would pass before phase 0)
          if (i == L::kESlots && !mbar_wait(smem_u32(&tail->dp_full), 0, abort_flag, a.dev_status))
            break;
          if (i >= L::kESlots &&
              !mbar_wait(smem_u32(&tail->dp_full), (i - 1) & 1, abort_flag, a.dev_status))
            break;
          const int s = i % L::kESlots;
          mbar_expect_tx(smem_u32(&tail->e_full[s]), L::kTileBytes);
          load(e_ring + s * L::kTileBytes, &p.m.d_o, tail->e_full[s],
               (begin + i % per_head) * kTile, g * a.group + i / per_head);
          ++ne;
          if (i + 1 < count) load_q(i + 1);
        }
        // copies in flight land before the CTA leaves
        mbar_wait_drain(smem_u32(&tail->k_full), 0);
        for (int s = 0; s < L::kQSlots && s < nq; ++s)
          mbar_wait_drain(smem_u32(&tail->q_full[s]), ((nq - 1 - s) / L::kQSlots) & 1);
        for (int s = 0; s < L::kESlots && s < ne; ++s)
          mbar_wait_drain(smem_u32(&tail->e_full[s]), ((ne - 1 - s) / L::kESlots) & 1);
      }
    } else if (warp == 9 && count > 0) {
      // ------------------------------------------------------ MMA
      const uint32_t on = elect_one();
      auto wait = [&](const uint64_t &bar, int phase) {  // one answer for the warp
        return wait_warp(bar, phase, abort_flag, a.dev_status);
      };
      auto padded = [&](int i) {
        return a.q_docs != nullptr && i < count &&
               doc_range(a.q_ranges, int64_t(b) * qtiles + begin + i % per_head).padded;
      };
      bool pads_q = padded(0), pads_e = pads_q;
      // a tile of step i has landed; without the rows of padding
      auto clear = [&](bool now, int tile, int i) {
        const int token = (begin + i % per_head) * kTile;
        if (now)
          zero_padding_rows<DH>(smem + tile * L::kTileBytes, a.q_docs + b * a.qds + token,
                                a.Sq - token);
      };
      auto wait_q = [&](int i) {
        const int s = i % L::kQSlots;
        if (!wait(tail->q_full[s], i / L::kQSlots)) return false;
        clear(pads_q, 2 + s, i);
        pads_q = padded(i + 1);
        return true;
      };
      auto wait_e = [&](int i) {
        const int s = i % L::kESlots;
        if (!wait(tail->e_full[s], i / L::kESlots)) return false;
        clear(pads_e, 2 + L::kQSlots + s, i);
        pads_e = padded(i + 1);
        return true;
      };
      auto q_at = [&](int i) { return q_ring + (i % L::kQSlots) * L::kTileBytes; };
      auto e_at = [&](int i) { return e_ring + (i % L::kESlots) * L::kTileBytes; };
      auto scores = [&](int i) {
        mma_over_head<DH>(on, tmem, k_tile, q_at(i));
        commit(on, smem_u32(&tail->s_full));
      };
      auto do_v = [&](int i) {
        mma_over_head<DH>(on, tmem + 128, v_tile, e_at(i));
        commit(on, smem_u32(&tail->dp_full));
      };
      bool ok = wait(tail->k_full, 0) && wait_q(0);
      tc_fence_after();
      if (ok) scores(0);
      if (ok) ok = wait_e(0);
      tc_fence_after();
      if (ok) do_v(0);
      for (int i = 0; i < count && ok; ++i) {
        if (!(ok = wait(tail->p_full, i))) break;
        tc_fence_after();
        mma_over_tokens<DH, 0, 8>(on, tmem + 256, tmem, operand_cols, e_at(i), i > 0);
        if (i + 1 < count) {  // over P^T, which the product before reads first
          if (!(ok = wait_q(i + 1))) break;
          tc_fence_after();
          scores(i + 1);
        }
        if (!(ok = wait(tail->dz_full, i))) break;
        tc_fence_after();
        mma_over_tokens<DH, 0, 8>(on, tmem + 384, tmem + 128, operand_cols, q_at(i), i > 0);
        if (i + 1 < count) {
          if (!(ok = wait_e(i + 1))) break;
          tc_fence_after();
          do_v(i + 1);
        }
        __syncwarp();
      }
      if (ok) commit(on, smem_u32(&tail->done));
      commit(on, smem_u32(&tail->drain));
      mbar_wait_drain(smem_u32(&tail->drain), 0);
      __syncwarp();
    }
  } else {
    set_max_regs_up<kPairRegs>();
    // ------------------------------------------------------ pairs
    const int half = warp / 4, r = threadIdx.x & 127, key = key0 + r;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + half * 64, dp_addr = s_addr + 128;
    // the first query that sees this key, and the last of the tile's keys
    const int from = a.causal && key >= prefix ? key - off : -(1 << 28);
    const int tile_last = key0 + kTile - 1;
    const int all_from = a.causal && tile_last >= prefix ? tile_last - off : -(1 << 28);
    const int kd = a.q_docs != nullptr && key < a.Sk ? a.k_docs[b * a.kds + key] : -1;
    // one of the two statistics of a query, fetched a step ahead: lse or delta
    const float *stat = (half == 0 ? a.lse : a.delta) + static_cast<int64_t>(b) * a.Hq * a.Sq;
    auto fetch = [&](int head, int n) {
      const int q = n * kTile + r;
      return q < a.Sq ? __ldcg(stat + static_cast<int64_t>(head) * a.Sq + q)
                      : half == 0 ? -INFINITY : 0.f;
    };
    auto put = [&](int i, float v) {
      if (half == 0)  // a query that sees nothing (lse = -inf): P = 0
        tail->sub[i & 1][r] = v == -INFINITY ? -INFINITY : -v * kLog2e;
      else
        tail->neg_delta[i & 1][r] = -v;
    };
    bool ok = true;
    DocRange qr = {0, 0, 0, 0};
    if (a.q_docs != nullptr && count > 0) qr = doc_range(a.q_ranges, int64_t(b) * qtiles + begin);
    if (count > 0) put(0, fetch(g * a.group, begin));
    int head = g * a.group, n = begin, head1 = head, n1 = begin;  // this step, the next
    for (int i = 0; i < count; ++i, head = head1, n = n1) {
      if (++n1 == end) {
        n1 = begin;
        ++head1;
      }
      const int q0 = n * kTile + half * 64;
      const ScoreConst sc = score_const(a, head);
      float ahead = 0.f;
      if (i + 1 < count) ahead = fetch(head1, n1);
      bool whole = n * kTile >= all_from;
      int qd[2];
      if (a.q_docs != nullptr) {
        whole = whole && docs_equal(kr, qr);
        if (!whole) load_docs(a.q_docs + b * a.qds + q0, a.Sq - q0, qd);
        if (i + 1 < count)
          qr = doc_range(a.q_ranges, int64_t(b) * qtiles + n1);
      }
      ok = ok && wait_warp(tail->s_full, i, abort_flag, a.dev_status);
      // everyone's statistics of this step are written, those of the step
      // before are no longer read
      if (!(ok = !named_bar_red_or(1, kPairThreads, !ok))) break;
      tc_fence_after();
      float w[64], pr[64];
      tmem_ld32(s_addr, w);
      tmem_ld32(s_addr + 32, w + 32);
      tmem_wait_ld();
      pin<64>(w);
      weights<CAP, BIAS, true>(sc, w, pr, 0.f, tail->sub[i & 1] + half * 64,
                               static_cast<float>(q0 + off - key), 1.f);
      if (!whole) {
        uint32_t keep[2] = {~0u, ~0u};
        if (a.q_docs != nullptr) same_doc(kd, qd, keep);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          keep[c] &= ~bits_to(from - 1 - q0 - 32 * c);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(keep[c] >> j & 1u)) w[c * 32 + j] = pr[c * 32 + j] = 0.f;
        }
      }
      {
        uint32_t z[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = pack_bf16(pr[2 * j], pr[2 * j + 1]);
        tmem_st16(s_addr, z);
        tmem_st16(s_addr + 16, z + 16);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&tail->p_full));
      if (i + 1 < count) put(i + 1, ahead);
      if (!(ok = wait_warp(tail->dp_full, i, abort_flag, a.dev_status))) continue;  // leave together, at the next barrier
      tc_fence_after();
      float dp[64];
      tmem_ld32(dp_addr, dp);
      tmem_ld32(dp_addr + 32, dp + 32);
      tmem_wait_ld();
      pin<64>(dp);
      const float *nd = tail->neg_delta[i & 1] + half * 64;
#pragma unroll
      for (int j = 0; j < 64; j += 4) {
        const float4 d = *reinterpret_cast<const float4 *>(nd + j);
        const float2 x = mul2(make_float2(w[j], w[j + 1]),
                              add2(make_float2(dp[j], dp[j + 1]), make_float2(d.x, d.y)));
        const float2 y = mul2(make_float2(w[j + 2], w[j + 3]),
                              add2(make_float2(dp[j + 2], dp[j + 3]), make_float2(d.z, d.w)));
        dp[j] = x.x;
        dp[j + 1] = x.y;
        dp[j + 2] = y.x;
        dp[j + 3] = y.y;
      }
      if (!whole) {  // a masked pair's dP and delta may be anything
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (w[j] == 0.f) dp[j] = 0.f;
      }
      uint32_t z[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) z[j] = pack_bf16(dp[2 * j], dp[2 * j + 1]);
      tmem_st16(dp_addr, z);
      tmem_st16(dp_addr + 16, z + 16);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&tail->dz_full));
    }
    if (ok && count > 0) {
      ok = wait_warp(tail->done, 0, abort_flag, a.dev_status);
    }
    // one warpgroup stages dk (in K's memory), the other dv (in V's)
    uint8_t *stage = smem + half * L::kTileBytes;
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < DH; c += 32) {
        float o[32];
        if (count > 0) {
          tmem_ld32(tmem + lanes + (half == 0 ? 384 : 256) + c, o);
          tmem_wait_ld();
          pin<32>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        stage_row32(stage, r, c, o, half == 0 ? a.scale : 1.f);
      }
      fence_proxy_async_smem();
    }
    const bool failed = named_bar_red_or(1, kPairThreads, !ok);
    if (!failed && r == 0) {
      for (int c = 0; c < DH / 64; ++c)
        if (c * 64 < a.D)
          tma_store_4d(half == 0 ? &p.m.dk : &p.m.dv, smem_u32(stage) + c * kTile * 128, c * 64,
                       key0, g, b);
      bulk_commit_group();
      bulk_wait_group0();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DH, bool CAP, bool BIAS>
cudaError_t start_dq(const Params &p, cudaStream_t s) {
  constexpr size_t smem = DqLayout<DH>::kAsked + sizeof(DqTail) + 1024;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_attn_dq<DH, CAP, BIAS>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(p.a.B) * p.a.Hq * ((p.a.Sq + kTile - 1) / kTile);
  return launch_pdl(k_attn_dq<DH, CAP, BIAS>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                    smem, s, p);
}
template <int DH, bool CAP, bool BIAS>
cudaError_t start_dkv(const Params &p, cudaStream_t s) {
  constexpr size_t smem = DkvLayout<DH>::kAsked;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_attn_dkv<DH, CAP, BIAS>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(p.a.B) * p.a.Hk * ((p.a.Sk + kTile - 1) / kTile);
  return launch_pdl(k_attn_dkv<DH, CAP, BIAS>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                    smem, s, p);
}

}  // namespace

#define LORA_ATTN_VARIANT(f)                                                            \
  const Params p{a, m};                                                                 \
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;                             \
  if (a.D <= 64)                                                                        \
    return cap ? (bias ? f<64, true, true>(p, s) : f<64, true, false>(p, s))            \
               : (bias ? f<64, false, true>(p, s) : f<64, false, false>(p, s));         \
  return cap ? (bias ? f<128, true, true>(p, s) : f<128, true, false>(p, s))            \
             : (bias ? f<128, false, true>(p, s) : f<128, false, false>(p, s))

cudaError_t launch_attn_dq(const AttnArgs &a, const AttnBwdMaps &m, cudaStream_t s) {
  LORA_ATTN_VARIANT(start_dq);
}
cudaError_t launch_attn_dkv(const AttnArgs &a, const AttnBwdMaps &m, cudaStream_t s) {
  LORA_ATTN_VARIANT(start_dkv);
}

}  // namespace lora
