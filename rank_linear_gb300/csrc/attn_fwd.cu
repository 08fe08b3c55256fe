// attn_fwd.cu -- attention forward on the tensor cores (include/lora_attention.h).
//
// A CTA takes 256 queries of one head as two tiles of 128 and passes once
// over the keys in tiles of 128: S = Q K^T into TMEM, softmax in registers (a
// thread owns a whole row: no shuffles), P back into TMEM as bf16 over S, and
// O += P V with P as the TMEM operand.  While the softmax of one tile runs,
// the tensor core works for the other.  The running maximum is only followed
// when it has moved by more than 2^8: until then P is relative to the old one
// (at most 256, exact in fp32 sums and no worse rounded to bf16), so that O
// in TMEM is hardly ever rescaled.
//
// TMEM: S/P of the two tiles at columns 0 and 128, O at 256 and 384.
#include "attn.cuh"
#include "host.h"

namespace lora {
namespace {

// Two softmax warpgroups, and one of which two warps issue the copies and the
// MMAs.  168 registers a thread at launch; the softmax threads, which hold a
// row of scores, take 224 and leave the others 56 (2 * 224 + 56 = 3 * 168).
constexpr int kThreads = 384, kSoftmaxRegs = 224, kIssueRegs = 56;
constexpr float kRescaleAt = 8.f;

template <int DH>
struct Layout {
  static constexpr uint32_t kTileBytes = kTile * DH * 2;
  // rings of K and V tiles; a V tile is asked for first and given back last
  static constexpr int kKSlots = DH == 64 ? 4 : 2, kVSlots = kKSlots + 1;
  static constexpr uint32_t kBytes = (2 + kKSlots + kVSlots) * kTileBytes;
};

struct Tail {
  uint64_t q_full, k_full[4], v_full[5];
  uint64_t passed[5];  // the products before step i, at i modulo kVSlots
  uint64_t s_full[2], p_full[2][2], o_done[2], drain;
  uint32_t tmem;
  int abort_flag;
  int lo[2], hi[2];
};

struct Params {
  AttnArgs a;
  AttnMaps m;
};

template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) k_attn_fwd(const __grid_constant__ Params p) {
  using L = Layout<DH>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Tail *tail = reinterpret_cast<Tail *>(smem + L::kBytes);
  const AttnArgs &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  // the blocks with most keys first: the last queries of a causal mask
  const int heads = a.B * a.Hq;
  const int blocks_q = (a.Sq + 2 * kTile - 1) / (2 * kTile);
  const int qb = blocks_q - 1 - static_cast<int>(blockIdx.x / heads);
  const int bh = blockIdx.x % heads, b = bh / a.Hq, h = bh % a.Hq, g = h / a.group;
  const int row0 = qb * 2 * kTile, off = a.Sk - a.Sq;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->q_full), 1);
    for (int s = 0; s < L::kKSlots; ++s) mbar_init(smem_u32(&tail->k_full[s]), 1);
    for (int s = 0; s < L::kVSlots; ++s) {
      mbar_init(smem_u32(&tail->v_full[s]), 1);
      mbar_init(smem_u32(&tail->passed[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&tail->s_full[t]), 1);
      mbar_init(smem_u32(&tail->p_full[t][0]), kTile);
      mbar_init(smem_u32(&tail->p_full[t][1]), kTile);
      mbar_init(smem_u32(&tail->o_done[t]), 1);
    }
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    for (int t = 0; t < 2; ++t) {
      tail->lo[t] = a.q_docs != nullptr ? INT_MAX : 0;
      tail->hi[t] = 0;
    }
    fence_barrier_init();
    tma_prefetch(&p.m.q);
    tma_prefetch(&p.m.k);
    tma_prefetch(&p.m.v);
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

  // ---- the key tiles [lo, hi) that some row of each query tile sees
  const int prefix = a.prefix != nullptr ? a.prefix[b] : 0;
  const int ktiles = (a.Sk + kTile - 1) / kTile, qtiles = (a.Sq + kTile - 1) / kTile;
  int most[2];
  for (int t = 0; t < 2; ++t) {
    const int first = row0 + t * kTile, last = min(first + kTile, a.Sq) - 1;
    most[t] = first < a.Sq ? (last_key(a, last + off, prefix) + kTile) / kTile : 0;
  }
  if (a.q_docs != nullptr) {
    for (int t = 0; t < 2; ++t) {
      if (most[t] <= 0) continue;
      const DocRange qr = doc_range(a.q_ranges, int64_t(b) * qtiles + 2 * qb + t);
      for (int n = threadIdx.x; n < most[t]; n += kThreads)
        if (docs_meet(qr, doc_range(a.k_ranges, int64_t(b) * ktiles + n))) {
          atomicMin(&tail->lo[t], n);
          atomicMax(&tail->hi[t], n + 1);
        }
    }
  } else if (threadIdx.x < 2) {
    tail->hi[threadIdx.x] = threadIdx.x == 0 ? most[0] : most[1];
  }
  __syncthreads();
  int lo[2], hi[2];
  for (int t = 0; t < 2; ++t) {
    hi[t] = uniform(max(tail->hi[t], 0));
    lo[t] = uniform(min(tail->lo[t], hi[t]));
  }
  // the tiles either passes over
  const int begin = hi[0] == lo[0] ? lo[1] : hi[1] == lo[1] ? lo[0] : min(lo[0], lo[1]);
  const int end = hi[0] == lo[0] ? hi[1] : hi[1] == lo[1] ? hi[0] : max(hi[0], hi[1]);

  // step i: P V of tile begin + i, and the scores of tile begin + i + 1
  const int count = end - begin;

  if (warp >= 8) {
    set_max_regs_down<kIssueRegs>();
    const uint32_t q_tile = smem_u32(smem), k_ring = q_tile + 2 * L::kTileBytes;
    const uint32_t v_ring = k_ring + L::kKSlots * L::kTileBytes;
    if (warp == 8) {
      // ------------------------------------------------------ TMA
      if (lane == 0 && count > 0) {
        auto load = [&](uint32_t dst, const CUtensorMap *tm, uint64_t &bar, int token, int head) {
          for (int c = 0; c < DH / 64; ++c)
            tma_load_4d(dst + c * kTile * 128, tm, smem_u32(&bar), c * 64, token, head, b);
        };
        auto load_k = [&](int i) {
          const int s = i % L::kKSlots;
          mbar_expect_tx(smem_u32(&tail->k_full[s]), L::kTileBytes);
          load(k_ring + s * L::kTileBytes, &p.m.k, tail->k_full[s], (begin + i) * kTile, g);
        };
        mbar_expect_tx(smem_u32(&tail->q_full), 2 * L::kTileBytes);
        for (int t = 0; t < 2; ++t)  // a second tile past the end reads as zeros
          load(q_tile + t * L::kTileBytes, &p.m.q, tail->q_full, row0 + t * kTile, h);
        load_k(0);
        int nk = 1, nv = 0;
        for (int i = 0; i < count; ++i) {
          const int s = i % L::kVSlots;
          mbar_expect_tx(smem_u32(&tail->v_full[s]), L::kTileBytes);
          load(v_ring + s * L::kTileBytes, &p.m.v, tail->v_full[s], (begin + i) * kTile, g);
          ++nv;
          if (i + 1 == count) break;
          // K's slot was scored before this step; so was V's next one
          const int gone = i + 1 - L::kKSlots;
          if (gone >= 0 && !mbar_wait(smem_u32(&tail->passed[gone % L::kVSlots]),
                                      (gone / L::kVSlots) & 1, abort_flag, a.dev_status))
            break;
          load_k(i + 1);
          ++nk;
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
      // (a commit holds the queue of MMAs for some 90 cycles: as few as will do)
      const uint32_t on = elect_one();
      auto wait = [&](const uint64_t &bar, int phase) {  // one answer for the warp
        return wait_warp(bar, phase, abort_flag, a.dev_status);
      };
      auto wait_k = [&](int i) { return wait(tail->k_full[i % L::kKSlots], i / L::kKSlots); };
      auto scores = [&](int t, int i) {
        mma_over_head<DH>(on, tmem + t * kTile, q_tile + t * L::kTileBytes,
                          k_ring + (i % L::kKSlots) * L::kTileBytes);
        commit(on, smem_u32(&tail->s_full[t]));
      };
      auto padded = [&](int i) {
        return a.q_docs != nullptr && i < count &&
               doc_range(a.k_ranges, int64_t(b) * ktiles + begin + i).padded;
      };
      const auto p_cols = [](int kk) { return kk * 8; };
      int turn[2] = {0, 0};  // score tiles done of each query tile
      // V's tile i has landed; without the rows of padding
      bool pads = padded(0);
      auto wait_v = [&](int i) {
        const int s = i % L::kVSlots, token = (begin + i) * kTile;
        if (!wait(tail->v_full[s], i / L::kVSlots)) return false;
        if (pads)
          zero_padding_rows<DH>(smem + (2 + L::kKSlots + s) * L::kTileBytes,
                                a.k_docs + b * a.kds + token, a.Sk - token);
        pads = padded(i + 1);
        return true;
      };
      bool ok = wait(tail->q_full, 0) && wait_k(0);
      tc_fence_after();
      if (ok)
        for (int t = 0; t < 2; ++t)
          if (begin >= lo[t] && begin < hi[t]) scores(t, 0);
      commit(on, smem_u32(&tail->passed[0]));
      if (ok) ok = wait_v(0);
      for (int i = 0; i < count && ok; ++i) {
        const int n = begin + i, vs = i % L::kVSlots;
        const bool more = i + 1 < count;
        const uint32_t vt = v_ring + vs * L::kTileBytes;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (n >= lo[t] && n < hi[t]) {
            const uint32_t o = tmem + 256 + t * kTile, w = tmem + t * kTile;
            if (!(ok = wait(tail->p_full[t][0], turn[t]))) break;
            tc_fence_after();
            mma_over_tokens<DH, 0, 4>(on, o, w, p_cols, vt, turn[t] > 0);
            if (!(ok = wait(tail->p_full[t][1], turn[t]))) break;
            tc_fence_after();
            mma_over_tokens<DH, 4, 8>(on, o, w, p_cols, vt, true);
            if (n + 1 == hi[t]) commit(on, smem_u32(&tail->o_done[t]));
            ++turn[t];
          }
          // While the queue is full: the step before is given back, and the
          // waits for what the next step reads.
          if (t == 0) {
            if (i > 0) commit(on, smem_u32(&tail->passed[vs]));
            if (more && !(ok = wait_k(i + 1))) break;
          } else if (more) {
            if (!(ok = wait_v(i + 1))) break;
          }
          tc_fence_after();
          if (n + 1 >= lo[t] && n + 1 < hi[t]) scores(t, i + 1);
        }
      }
      // nothing of this CTA is in flight when it leaves
      commit(on, smem_u32(&tail->drain));
      mbar_wait_drain(smem_u32(&tail->drain), 0);
      __syncwarp();
    }
  } else {
    set_max_regs_up<kSoftmaxRegs>();
    // ------------------------------------------------------ softmax
    const int t = warp / 4;
    const int row = row0 + t * kTile + (threadIdx.x & 127);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * kTile, o_addr = tmem + lanes + 256 + t * kTile;
    const ScoreConst sc = score_const(a, h);
    const int pos = row + off;
    const int last = row < a.Sq ? last_key(a, pos, prefix) : -1;
    const int first_last = last_key(a, row0 + t * kTile + off, prefix);  // of the tile's first row
    DocRange qr = {0, 0, 0, 0};
    int qd = 0;
    if (a.q_docs != nullptr && row0 + t * kTile < a.Sq) {
      qr = doc_range(a.q_ranges, int64_t(b) * qtiles + 2 * qb + t);
      qd = row < a.Sq ? a.q_docs[b * a.qds + row] : -1;
    }
    float m = -INFINITY;  // the maximum that P is relative to, in log2 units
    float2 l2 = make_float2(0.f, 0.f);
    bool ok = true;
    int turn = 0;
    DocRange kr = {0, 0, 0, 0};
    if (a.q_docs != nullptr && lo[t] < hi[t])
      kr = doc_range(a.k_ranges, int64_t(b) * ktiles + lo[t]);
    for (int n = lo[t]; n < hi[t]; ++n, ++turn) {
      // does the mask leave the whole tile?
      bool whole = n * kTile + kTile - 1 <= first_last;
      int kd[4];
      if (a.q_docs != nullptr) {
        whole = whole && docs_equal(qr, kr);
        if (!whole) load_docs(a.k_docs + b * a.kds + n * kTile, a.Sk - n * kTile, kd);
        if (n + 1 < hi[t]) kr = doc_range(a.k_ranges, int64_t(b) * ktiles + n + 1);
      }
      if (!(ok = wait_warp(tail->s_full[t], turn, abort_flag, a.dev_status))) break;
      tc_fence_after();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, s + c * 32);
      tmem_wait_ld();
      pin<kTile>(s);
      if constexpr (CAP || BIAS) {
        const float d0 = static_cast<float>(pos - n * kTile);
        float r;
#pragma unroll
        for (int j = 0; j < kTile; ++j) s[j] = score2<CAP, BIAS>(sc, s[j], d0 - j, r);
      }
      if (!whole) {
        uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
        if (a.q_docs != nullptr) same_doc(qd, kd, keep);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          keep[c] &= bits_to(last - n * kTile - 32 * c);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(keep[c] >> j & 1u)) s[c * 32 + j] = -INFINITY;
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int j = 4; j < kTile - 4; j += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[j + 2 * i], s[j + 2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], s[kTile - 4 + i]);
      float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      if constexpr (!CAP && !BIAS) top *= sc.scale2;
      float by = 1.f;
      if (m == -INFINITY) {
        m = top;  // nothing summed so far: O's row is zero or not begun
      } else if (top > m + kRescaleAt) {
        by = ex2(m - top);
        m = top;
      }
      if (__any_sync(~0u, by != 1.f)) {
        // (the scores of this tile were issued after P V of the one before:
        // that is in O)
        l2.x *= by;
        l2.y *= by;
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          float o[32];
          tmem_ld32(o_addr + c, o);
          tmem_wait_ld();
          pin<32>(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= by;
          tmem_st32(o_addr + c, o);
        }
      }
      const float sub = m == -INFINITY ? 0.f : -m;
      const float2 sub2 = make_float2(sub, sub);
      const float2 sl2 = make_float2(sc.scale2, sc.scale2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 x = make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]);
          if constexpr (CAP || BIAS)
            x = add2(x, sub2);
          else
            x = fma2(x, sl2, sub2);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          l2 = add2(l2, x);
          w[i] = pack_bf16(x.x, x.y);
        }
        tmem_st16(s_addr + c * 16, w);
        if (c & 1) {  // P V may begin on the first half
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(&tail->p_full[t][c >> 1]));
        }
      }
    }
    if (row0 + t * kTile < a.Sq) {
      if (ok && turn > 0) {
        ok = wait_warp(tail->o_done[t], 0, abort_flag, a.dev_status);
      } else if (ok && count > 0) {  // Q's copy has landed before its memory is reused
        ok = wait_warp(tail->q_full, 0, abort_flag, a.dev_status);
      }
      const float l = l2.x + l2.y;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (ok) {
        // O through this tile's part of Q's shared memory: every product that
        // reads it is done
        tc_fence_after();
        uint8_t *stage = smem + t * L::kTileBytes;
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          float o[32];
          if (turn > 0) {
            tmem_ld32(o_addr + c, o);
            tmem_wait_ld();
            pin<32>(o);
          }
          if (!(l > 0.f))
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          stage_row32(stage, threadIdx.x & 127, c, o, inv);
        }
        if (a.lse != nullptr && row < a.Sq)
          a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Sq + row] =
              l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
        fence_proxy_async_smem();
      }
      // stored only if every warp of the tile has its rows staged
      const bool failed = named_bar_red_or(1 + t, kTile, !ok);
      if (!failed) {
        uint8_t *stage = smem + t * L::kTileBytes;
        if ((threadIdx.x & 127) == 0) {
          for (int c = 0; c < DH / 64; ++c)
            if (c * 64 < a.D)
              tma_store_4d(&p.m.o, smem_u32(stage) + c * kTile * 128, c * 64, row0 + t * kTile, h, b);
          bulk_commit_group();
          bulk_wait_group0();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Ranges of the documents of 128-token tiles, one warp per tile.
__global__ void k_attn_ranges(const int *docs, int64_t stride, int B, int S, int4 *out) {
  griddep_wait();
  griddep_launch_dependents();
  const int tiles = (S + kTile - 1) / kTile;
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
  if (w >= B * tiles) return;
  const int b = w / tiles, n = w % tiles;
  int lo = INT_MAX, hi = -1, padded = 0;
  for (int i = lane; i < kTile; i += 32) {
    const int at = n * kTile + i;
    if (at >= S) break;
    const int d = docs[b * stride + at];
    if (d < 0) {
      padded = 1;
    } else {
      lo = min(lo, d);
      hi = max(hi, d);
    }
  }
  lo = __reduce_min_sync(~0u, lo);
  hi = __reduce_max_sync(~0u, hi);
  padded = __any_sync(~0u, padded);
  if (lane == 0) out[w] = make_int4(lo, hi, padded, 0);
}

template <int DH, bool CAP, bool BIAS>
cudaError_t launch(const Params &p, cudaStream_t s) {
  const size_t smem = Layout<DH>::kBytes + sizeof(Tail) + 1024;
  auto *kernel = k_attn_fwd<DH, CAP, BIAS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = int64_t(p.a.B) * p.a.Hq * ((p.a.Sq + 2 * kTile - 1) / (2 * kTile));
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_attn_ranges(const AttnArgs &a, cudaStream_t s) {
  for (int side = 0; side < 2; ++side) {
    const int S = side ? a.Sk : a.Sq;
    const int64_t tiles = int64_t(a.B) * ((S + kTile - 1) / kTile);
    if (tiles == 0) continue;
    const cudaError_t e = launch_pdl(
        k_attn_ranges, dim3(static_cast<unsigned>((tiles + 7) / 8)), dim3(256), 0, s,
        side ? a.k_docs : a.q_docs, side ? a.kds : a.qds, a.B, S,
        const_cast<int4 *>(side ? a.k_ranges : a.q_ranges));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_attn_fwd(const AttnArgs &a, const AttnMaps &m, cudaStream_t s) {
  const Params p{a, m};
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  if (a.D <= 64)
    return cap ? (bias ? launch<64, true, true>(p, s) : launch<64, true, false>(p, s))
               : (bias ? launch<64, false, true>(p, s) : launch<64, false, false>(p, s));
  return cap ? (bias ? launch<128, true, true>(p, s) : launch<128, true, false>(p, s))
             : (bias ? launch<128, false, true>(p, s) : launch<128, false, false>(p, s));
}

}  // namespace lora
