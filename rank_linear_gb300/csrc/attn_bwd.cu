// attn_bwd.cu -- attention backward on the tensor cores (include/lora_attention.h).
//
// Two kernels, so that every sum has one owner and a fixed order (no atomics):
// one passes over the keys for 128 queries and keeps dq in TMEM, the other
// over the queries of all heads of a group for 128 keys and keeps dk and dv.
// Each recomputes the scores, seven products of 128 x 128 tiles in all where
// sharing them across blocks would take five.  What a thread computes for a
// pair, dz = P dc/dz (dP - delta) with P = exp(s - lse), goes back into TMEM
// as bf16 over the scores (or over dP) and is the TMEM operand of the products
// that follow; nothing of size q_len x k_len leaves the SM.  That rounding of
// dz, and of P for dv, costs what the outputs' own does, 0.0017 of their norm
// each; two bf16 parts of dz would be nine products instead of seven.
//
// A small pass before them leaves two numbers of each query row, -lse in log2
// units and -delta = -do . o, in rows of whole tiles: read once for both
// kernels.  (Formed in the dq kernel they cost an item 3600 to 10000 cycles,
// or 22000 of the first one in warps of their own.)  o there has been rounded
// to bf16, which is most of the error of a gradient that nearly cancels: with
// few keys, a query that looks almost wholly at one of them (of two keys dq is
// off by 0.006 of its norm in the median, by 0.2 in a row of ten).  Rows whose
// keys lie in one tile therefore have delta = sum_j P dP formed in the dq
// kernel, whose tile has both, and left for dk and dv: the first rows of a
// causal mask, short documents, and whatever looks at 128 keys or fewer.  It is
// a pass of its own over such tiles, which are few, so that the registers and
// the code of the others stay as they are (in one pass, heads of 64 causal at
// 8192: dq 430 us; in two, 418; without, 400), and only where the mask may
// leave some row no other tile (of five documents in 8192: dq 199 us over the
// last tile of every item, 187 so, 181 without).  Rows that see more keep delta
// from o: for them it would take the scores of all their tiles twice.
//
// The dq blocks stay and take item after item, as the forward's do.  A dk/dv
// item has a group's heads times as much work; where there are too few for the
// SMs, the blocks of a cluster share one, each with its part of the steps, and
// add their sums through distributed shared memory in the order of their ranks.
//
// Measured (32 heads of 128, 8 key heads), all three: 8192 x 8192 without a
// mask 2502 us (1100 TFLOP/s of the formula's five products, 1540 of the seven
// done), causal 1202 us (1145), 4096 causal 337 us (1020), with a cap 478 us,
// five documents in 8192 466 us, five others 481 us (statistics 27, dq 186,
// dk/dv 260 when timed one by one), heads of 64 causal 1007 us (680: the
// exponentials twice more, and half the products to set against them).  Bound
// by shared memory: a dk/dv step's products read 256 KB of operands, 2000
// cycles at 128 B a cycle, as long as the products themselves take.
#include "attn.cuh"
#include "host.h"

namespace lora {
namespace {

// Two warpgroups for the pairs (128 rows, 64 columns each) and one whose warps
// issue the copies, the MMAs and the items; registers as in the forward.
constexpr int kThreads = 384, kPairThreads = 256, kPairRegs = 224, kIssueRegs = 56;
constexpr int kItemSlots = 2, kItemReaders = 10;

struct Params {
  AttnArgs a;
  AttnBwdMaps m;
  int items, cluster;
};

// The columns of a 128-wide TMEM region that hold K step kk of a bf16 operand:
// the warpgroup of columns 0..63 writes columns 0..31, the other 64..95, each
// over scores that it alone reads.
__device__ __forceinline__ constexpr uint32_t operand_cols(int kk) { return (kk >> 2) * 64 + (kk & 3) * 8; }

// P (to p) and P dc/dz / scale (in s) of N raw products of one thread;
// distances d0 + step * j; sub = -lse in log2 units (or one per column in
// sub_col).
template <bool CAP, bool BIAS, bool PER_COLUMN, int N>
__device__ __forceinline__ void weights(const ScoreConst &c, float (&s)[N], float *p, float sub,
                                        const float *sub_col, float d0, float step) {
  auto all = [&](bool small) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
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
        float2 f = make_float2(1.f, 1.f);
        if constexpr (CAP || BIAS) {
          float2 t = x;  // tanh: 1 - t^2 is its slope
          if constexpr (CAP) {
            if (small) {
              t = cap_small(c, x);
              f = fma2(make_float2(-t.x, -t.y), t, f);
            } else {
              t = cap_near(c, x);
              const float2 r = make_float2(cap_r(c, fabsf(x.x)), cap_r(c, fabsf(x.y)));
              t = make_float2(copysignf(cap_any(c, x.x, r.x, t.x), x.x),
                              copysignf(cap_any(c, x.y, r.y, t.y), x.y));
              f = make_float2(4.f * r.x * (1.f - r.x), 4.f * r.y * (1.f - r.y));
            }
          }
          const float by = CAP ? c.cap2 : c.scale2;
          x = mul2(t, make_float2(by, by));
          if constexpr (BIAS) {
            const float d = d0 + step * (j + i);
            x.x = fmaf(-c.slope2, fabsf(d), x.x);
            x.y = fmaf(-c.slope2, fabsf(d + step), x.y);
          }
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
        if constexpr (CAP) x = mul2(x, f);
        s[j + i] = x.x;
        s[j + i + 1] = x.y;
      }
    }
  };
  if (!CAP || all_small<N>(c, s))
    all(true);
  else
    all(false);
}

// ---------------------------------------------------------------- statistics
// A warp takes 32 queries of one head (its neighbours the next heads, which
// lie beside it), DH / 8 lanes to a row.  Bound by HBM and its few waves: 8192
// queries of 32 heads of 128, 134 MB, 28 us from a cold L2.
constexpr int kStatWarps = 8;
template <int DH>
__global__ void __launch_bounds__(32 * kStatWarps) k_attn_stats(const AttnArgs a) {
  constexpr int kLanes = DH / 8, kRows = 32 / kLanes, kLoads = 8;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32, groups = (a.Hq + kStatWarps - 1) / kStatWarps;
  const int padded = (a.Sq + kTile - 1) / kTile * kTile, blocks = padded / 32;
  int id = blockIdx.x;
  const int h = id % groups * kStatWarps + threadIdx.x / 32;
  id /= groups;
  const int row0 = id % blocks * 32, b = id / blocks;
  if (h >= a.Hq) return;
  const int e = lane % kLanes * 8;
  const __nv_bfloat16 *o =
      static_cast<const __nv_bfloat16 *>(a.o) + b * a.so[0] + h * a.so[2] + e;
  const __nv_bfloat16 *g =
      static_cast<const __nv_bfloat16 *>(a.d_o) + b * a.sdo[0] + h * a.sdo[2] + e;
  const int64_t row = static_cast<int64_t>(b) * a.Hq + h;
  float lse = -INFINITY, delta = 0.f;  // of query row0 + lane
  if (row0 + lane < a.Sq) lse = __ldcg(a.lse + row * a.Sq + row0 + lane);
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += kLoads * kRows) {
    uint4 xo[kLoads], xg[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t at = row0 + r0 + i * kRows + lane / kLanes;
      xo[i] = xg[i] = make_uint4(0, 0, 0, 0);
      if (at < a.Sq && e < a.D) {
        xo[i] = __ldcg(reinterpret_cast<const uint4 *>(o + at * a.so[1]));
        xg[i] = __ldcg(reinterpret_cast<const uint4 *>(g + at * a.sdo[1]));
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t u[4] = {xo[i].x, xo[i].y, xo[i].z, xo[i].w};
      const uint32_t v[4] = {xg[i].x, xg[i].y, xg[i].z, xg[i].w};
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        d = fmaf(__uint_as_float(u[k] << 16), __uint_as_float(v[k] << 16), d);
        d = fmaf(__uint_as_float(u[k] & 0xffff0000u), __uint_as_float(v[k] & 0xffff0000u), d);
      }
#pragma unroll
      for (int y = 1; y < kLanes; y *= 2) d += __shfl_xor_sync(~0u, d, y);
      // row r0 + i kRows + j is in the lanes of group j: hand it to its owner
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const float x = __shfl_sync(~0u, d, j * kLanes);
        if (lane == r0 + i * kRows + j) delta = x;
      }
    }
  }
  const int64_t at = row * padded + row0 + lane;
  // a query that sees nothing, or lies past the end: P = 0
  a.sub[at] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
  a.neg_delta[at] = -delta;
}

// ---------------------------------------------------------------- dq
// Shared memory: Q, dO, then rings of K and V tiles (counted on over the items).  TMEM: the scores (then
// dz) of two tiles at 0 and 128, dP at 256, dq at 384.
template <int DH>
struct DqLayout {
  static constexpr uint32_t kTileBytes = kTile * DH * 2;
  static constexpr int kKSlots = 3, kVSlots = 2;
  // the tiles follow the tail (DqTail), which for a head of 128 fills what
  // they leave of an SM's 227 KB: no room to align a base that is not aligned
  static constexpr uint32_t kTailBytes = 3072;
  static constexpr uint32_t kBytes = kTailBytes + (2 + kKSlots + kVSlots) * kTileBytes;
  // one block per SM (TMEM): more than half of its shared memory
  static constexpr uint32_t kAsked = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
// 128 queries from row0 of head h, batch entry b, and the key tiles [begin,
// begin + count) that some row sees.  count < 0: no more items.
struct DqItem {
  int row0, h, b, begin, count;
  int same[2];  // key tiles [0], ..., [1] - 1 of the queries' one document
};
struct DqTail {
  uint64_t q_full, q_free, k_full[3], k_empty[3], v_full[2];
  uint64_t s_full[2], dp_full[2], dp_free, done, drain;
  uint64_t dz_full[2];  // by tile modulo 2: tile x + 1's may come before x's is waited for
  uint64_t item_full[kItemSlots], item_free[kItemSlots];
  uint64_t own;            // a half row's sums are there, then: they have been read
  float2 part[2][kTile];   // sums of P and of P dP in a tile, of each half
  DqItem item[kItemSlots];
  uint32_t tmem;
  int abort_flag;
};

__device__ __forceinline__ bool next_item(DqTail *tail, int n, DqItem &item,
                                          volatile int *abort_flag, unsigned *dev_status) {
  const int s = n % kItemSlots;
  if (!wait_warp(tail->item_full[s], n / kItemSlots, abort_flag, dev_status)) return false;
  item = tail->item[s];
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(smem_u32(&tail->item_free[s]));
  return item.count >= 0;
}

template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) k_attn_dq(const __grid_constant__ Params p) {
  using L = DqLayout<DH>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t *smem = raw + L::kTailBytes;
  DqTail *tail = reinterpret_cast<DqTail *>(raw);
  static_assert(sizeof(DqTail) <= L::kTailBytes, "tail");
  if ((smem_u32(raw) & 1023) != 0) {  // not met: the tiles' layout needs it
    if (threadIdx.x == 0) atomicOr(p.a.dev_status, kDevErrTimeout);
    return;
  }
  const AttnArgs &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int off = a.Sk - a.Sq;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->q_full), 1);
    mbar_init(smem_u32(&tail->q_free), 1);
    for (int s = 0; s < L::kKSlots; ++s) {
      mbar_init(smem_u32(&tail->k_full[s]), 1);
      mbar_init(smem_u32(&tail->k_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&tail->v_full[s]), 1);
      mbar_init(smem_u32(&tail->s_full[s]), 1);
      mbar_init(smem_u32(&tail->dp_full[s]), 1);
      mbar_init(smem_u32(&tail->dz_full[s]), kPairThreads);
    }
    mbar_init(smem_u32(&tail->dp_free), kPairThreads);
    mbar_init(smem_u32(&tail->own), kPairThreads);
    for (int s = 0; s < kItemSlots; ++s) {
      mbar_init(smem_u32(&tail->item_full[s]), 1);
      mbar_init(smem_u32(&tail->item_free[s]), kItemReaders);
    }
    mbar_init(smem_u32(&tail->done), 1);
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
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

  if (warp >= 8) {
    set_max_regs_down<kIssueRegs>();
    const uint32_t q_tile = smem_u32(smem), do_tile = q_tile + L::kTileBytes;
    const uint32_t k_ring = do_tile + L::kTileBytes, v_ring = k_ring + L::kKSlots * L::kTileBytes;
    auto wait = [&](const uint64_t &bar, int phase) {
      return wait_warp(bar, phase, abort_flag, a.dev_status);
    };
    if (warp == 10) {
      // ------------------------------------------------------ items
      const int heads = a.B * a.Hq;
      for (int n = 0;; ++n) {
        const int s = n % kItemSlots;
        if (n >= kItemSlots && !wait(tail->item_free[s], n / kItemSlots - 1)) break;
        // to and fro over the blocks, or from the counter, as in the forward
        const int blocks = gridDim.x, place = blockIdx.x;
        int id = n * blocks + (n & 1 ? blocks - 1 - place : place);
        if (a.counter != nullptr && n > 0) {
          if (lane == 0) id = blocks + static_cast<int>(atomicAdd(a.counter, 1u));
          id = __shfl_sync(~0u, id, 0);
        }
        DqItem it = {};
        it.count = -1;
        if (id < p.items) {
          const int qt = qtiles - 1 - id / heads, bh = id % heads;
          it.b = bh / a.Hq;
          it.h = bh % a.Hq;
          it.row0 = qt * kTile;
          const int prefix = a.prefix != nullptr ? a.prefix[it.b] : 0;
          int lo = 0, hi = max(0, (last_key(a, min(it.row0 + kTile, a.Sq) - 1 + off, prefix) +
                                   kTile) / kTile);
          it.same[0] = 0;
          it.same[1] = INT_MAX;  // no documents: one
          if (a.q_docs != nullptr && hi > 0)
            doc_tiles(doc_range(a.q_ranges, int64_t(it.b) * qtiles + qt),
                      a.k_ranges + int64_t(it.b) * ktiles, lo, hi, it.same);
          it.begin = lo;
          it.count = hi - lo;
        }
        if (lane == 0) {
          tail->item[s] = it;
          mbar_arrive(smem_u32(&tail->item_full[s]));  // releases the item's words
          if (it.count > 0)  // what it begins with, towards L2
            for (int c = 0; c < DH; c += 64) {
              tma_prefetch_4d(&p.m.q, c, it.row0, it.h, it.b);
              tma_prefetch_4d(&p.m.d_o, c, it.row0, it.h, it.b);
              tma_prefetch_4d(&p.m.k, c, it.begin * kTile, it.h / a.group, it.b);
              tma_prefetch_4d(&p.m.v, c, it.begin * kTile, it.h / a.group, it.b);
            }
        }
        __syncwarp();
        if (it.count < 0) break;
      }
    } else if (warp == 8) {
      // ------------------------------------------------------ TMA
      int x = 0, used = 0, nv = 0;  // tiles loaded so far, items with tiles
      bool ok = true;
      DqItem it;
      for (int n = 0; ok && next_item(tail, n, it, abort_flag, a.dev_status); ++n) {
        if (it.count == 0) continue;
        if (used > 0 && !(ok = wait(tail->q_free, used - 1))) break;
        const int g = it.h / a.group;
        auto load = [&](uint32_t dst, const CUtensorMap *tm, uint64_t &bar, int token, int head) {
          for (int c = 0; c < DH / 64; ++c)
            tma_load_4d(dst + c * kTile * 128, tm, smem_u32(&bar), c * 64, token, head, it.b);
        };
        if (lane == 0) {
          mbar_expect_tx(smem_u32(&tail->q_full), 2 * L::kTileBytes);
          load(q_tile, &p.m.q, tail->q_full, it.row0, it.h);
          load(do_tile, &p.m.d_o, tail->q_full, it.row0, it.h);
        }
        ++used;
        for (int i = 0; i < it.count; ++i, ++x) {
          const int ks = x % L::kKSlots, vs = x % L::kVSlots, token = (it.begin + i) * kTile;
          if (x >= L::kKSlots && !(ok = wait(tail->k_empty[ks], x / L::kKSlots - 1))) break;
          if (lane == 0) {
            mbar_expect_tx(smem_u32(&tail->k_full[ks]), L::kTileBytes);
            load(k_ring + ks * L::kTileBytes, &p.m.k, tail->k_full[ks], token, g);
          }
          // dP of the tile before in this slot is done
          if (x >= L::kVSlots && !(ok = wait(tail->dp_full[vs], x / L::kVSlots - 1))) {
            ++x;  // K's copy alone is in flight
            break;
          }
          if (lane == 0) {
            mbar_expect_tx(smem_u32(&tail->v_full[vs]), L::kTileBytes);
            load(v_ring + vs * L::kTileBytes, &p.m.v, tail->v_full[vs], token, g);
          }
          ++nv;
          __syncwarp();
        }
      }
      // copies in flight land before the CTA leaves
      if (lane == 0) {
        if (used > 0) mbar_wait_drain(smem_u32(&tail->q_full), (used - 1) & 1);
        for (int s = 0; s < L::kKSlots && s < x; ++s)
          mbar_wait_drain(smem_u32(&tail->k_full[s]), ((x - 1 - s) / L::kKSlots) & 1);
        for (int s = 0; s < L::kVSlots && s < nv; ++s)
          mbar_wait_drain(smem_u32(&tail->v_full[s]), ((nv - 1 - s) / L::kVSlots) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------ MMA
      const uint32_t on = elect_one();
      int base = 0, used = 0;  // tiles and items with tiles before this item
      bool ok = true;
      DqItem it;
      for (int n = 0; ok && next_item(tail, n, it, abort_flag, a.dev_status); ++n) {
        const int count = uniform(it.count), begin = uniform(it.begin), b = uniform(it.b);
        if (count == 0) continue;
        auto padded = [&](int i) {
          return a.q_docs != nullptr && i < count
                     ? doc_range(a.k_ranges, int64_t(b) * ktiles + begin + i).padded
                     : 0;
        };
        // K's tile i has landed, without the rows of padding
        int pads = padded(0);  // looked at a step later: not waited for here
        auto wait_k = [&](int i) {
          const int s = (base + i) % L::kKSlots, token = (begin + i) * kTile;
          if (!wait(tail->k_full[s], (base + i) / L::kKSlots)) return false;
          const int now = pads;
          pads = padded(i + 1);
          if (now != 0)
            zero_padding_rows<DH>(smem + (2 + s) * L::kTileBytes, a.k_docs + b * a.kds + token,
                                  a.Sk - token);
          return true;
        };
        auto scores = [&](int i) {
          const int x = base + i;
          mma_over_head<DH>(on, tmem + (x & 1) * kTile, q_tile,
                            k_ring + (x % L::kKSlots) * L::kTileBytes);
          commit(on, smem_u32(&tail->s_full[x & 1]));
        };
        // V's tile has landed, dP of the tile before is in registers
        auto wait_v = [&](int i) {
          const int x = base + i;
          return wait(tail->v_full[x % L::kVSlots], x / L::kVSlots) &&
                 (x == 0 || wait(tail->dp_free, x - 1));
        };
        auto do_v = [&](int i) {
          const int x = base + i;
          mma_over_head<DH>(on, tmem + 256, do_tile, v_ring + (x % L::kVSlots) * L::kTileBytes);
          commit(on, smem_u32(&tail->dp_full[x % L::kVSlots]));
          if (i + 1 == count) commit(on, smem_u32(&tail->q_free));  // Q and dO have been read
        };
        if (!(ok = wait(tail->q_full, used) && wait_k(0))) break;
        tc_fence_after();
        scores(0);
        if (!(ok = wait_v(0))) break;
        tc_fence_after();
        do_v(0);
        for (int i = 0; i < count; ++i) {
          const int x = base + i;
          if (i + 1 < count) {
            // over the dz of tile i - 1, which its product (issued) reads first
            if (!(ok = wait_k(i + 1))) break;
            tc_fence_after();
            scores(i + 1);
            if (!(ok = wait_v(i + 1))) break;
            tc_fence_after();
            do_v(i + 1);
          }
          if (!(ok = wait(tail->dz_full[x & 1], x >> 1))) break;
          tc_fence_after();
          mma_over_tokens<DH, 0, 8>(on, tmem + 384, tmem + (x & 1) * kTile, operand_cols,
                                    k_ring + (x % L::kKSlots) * L::kTileBytes, i > 0);
          commit(on, smem_u32(&tail->k_empty[x % L::kKSlots]));
        }
        if (ok) commit(on, smem_u32(&tail->done));
        base += count;
        ++used;
      }
      commit(on, smem_u32(&tail->drain));
      mbar_wait_drain(smem_u32(&tail->drain), 0);
      __syncwarp();
    }
  } else {
    set_max_regs_up<kPairRegs>();
    // ------------------------------------------------------ pairs
    const int half = warp / 4, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int x = 0, used = 0;  // tiles, and items with tiles, before this one
    int owned = 0;        // tiles whose sums were shared before this one
    bool ok = true;
    // an item, and what is read for its row: asked for before the item ahead
    // of it is written out
    DqItem it;
    float sub = 0.f, neg_delta = 0.f;
    int prefix = 0, qd = -1;
    auto take = [&](int n) {
      if (!next_item(tail, n, it, abort_flag, a.dev_status)) return false;
      const int64_t at = (static_cast<int64_t>(it.b) * a.Hq + it.h) * (qtiles * kTile) + it.row0 + r;
      sub = __ldcg(a.sub + at);
      neg_delta = __ldcg(a.neg_delta + at);
      if (a.prefix != nullptr) prefix = a.prefix[it.b];
      if (a.q_docs != nullptr)
        qd = it.row0 + r < a.Sq ? a.q_docs[it.b * a.qds + it.row0 + r] : -1;
      return true;
    };
    bool more = take(0);
    for (int item = 0; more; ++item) {
      const int b = it.b, h = it.h, row = it.row0 + r, count = it.count;
      const ScoreConst sc = score_const(a, h, true);
      const int pos = row + off;
      const int last = row < a.Sq ? last_key(a, pos, prefix) : -1;
      const int first_last = last_key(a, it.row0 + off, prefix);
      const int same0 = it.same[0], same1 = it.same[1], begin = it.begin;
      for (int i = 0; i < count; ++i, ++x) {
        const int n = begin + i, key0 = n * kTile + half * 64;
        const bool same = n >= same0 && n < same1;
        const bool whole = same && n * kTile + kTile - 1 <= first_last;
        int kd[2];
        if (!same) load_docs(a.k_docs + b * a.kds + key0, a.Sk - key0, kd);
        const uint32_t s_addr = tmem + lanes + (x & 1) * kTile + half * 64;
        const uint32_t dp_addr = tmem + lanes + 256 + half * 64;
        if (!(ok = wait_warp(tail->s_full[x & 1], x >> 1, abort_flag, a.dev_status))) break;
        // May some row see this tile's keys only?  (Of a causal mask each row
        // sees itself: in a tile that reaches the first row's place.  Not where
        // every row sees all of another tile.)
        const bool close = a.q_docs == nullptr ? n == 0 && first_last < kTile
                           : count == 1 ||
                                 ((a.causal && a.prefix == nullptr ? n * kTile + kTile > first_last
                                                                   : !whole) &&
                                  (n == same0 || same0 >= same1 ||
                                   same0 * kTile + kTile - 1 > first_last));
        if (close) {  // a pass of its own, so that the other tiles' registers stay as they are
          if (!(ok = wait_warp(tail->dp_full[x & 1], x >> 1, abort_flag, a.dev_status))) break;
          tc_fence_after();
          uint32_t keep[2] = {~0u, ~0u};
          if (!same) same_doc(qd, kd, keep);
          float2 all = make_float2(0.f, 0.f), sum = all;  // of P, of P dP
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            float w[32], pr[32], dp[32];
            tmem_ld32(s_addr + c, w);
            tmem_ld32(dp_addr + c, dp);
            tmem_wait_ld();
            pin<32>(w);
            pin<32>(dp);
            weights<CAP, BIAS, false>(sc, w, pr, sub, nullptr, static_cast<float>(pos - key0 - c),
                                      -1.f);
            const uint32_t see = (c == 0 ? keep[0] : keep[1]) & bits_to(last - key0 - c);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {  // (a masked pair's dP may be anything)
              const bool one = see >> j & 1u, two = see >> j & 2u;
              const float2 y = make_float2(one ? pr[j] : 0.f, two ? pr[j + 1] : 0.f);
              all = add2(all, y);
              sum = fma2(y, make_float2(one ? dp[j] : 0.f, two ? dp[j + 1] : 0.f), sum);
            }
          }
          if (owned > 0 && !(ok = wait_warp(tail->own, 2 * owned - 1, abort_flag, a.dev_status)))
            break;
          tail->part[half][r] = make_float2(all.x + all.y, sum.x + sum.y);
          mbar_arrive(smem_u32(&tail->own));
          if (!(ok = wait_warp(tail->own, 2 * owned, abort_flag, a.dev_status))) break;
          const float2 one = tail->part[0][r], two = tail->part[1][r];
          mbar_arrive(smem_u32(&tail->own));
          ++owned;
          // by the mask; with documents by the weight (what is left of it is
          // less than 2^-12, and moves delta by that of what dP differs)
          if (a.q_docs != nullptr ? one.x + two.x >= 1.f - 0x1p-12f : last < kTile) {
            neg_delta = -(one.y + two.y);
            if (half == 0)
              a.neg_delta[(static_cast<int64_t>(b) * a.Hq + h) * (qtiles * kTile) + row] = neg_delta;
          }
        }
        tc_fence_after();
        float w[64];
        tmem_ld32(s_addr, w);
        tmem_ld32(s_addr + 32, w + 32);
        tmem_wait_ld();
        pin<64>(w);
        weights<CAP, BIAS, false>(sc, w, nullptr, sub, nullptr,
                                  static_cast<float>(pos - key0), -1.f);
        if (!whole) {
          uint32_t keep[2] = {~0u, ~0u};
          if (!same) same_doc(qd, kd, keep);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            keep[c] &= bits_to(last - key0 - 32 * c);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(keep[c] >> j & 1u)) w[c * 32 + j] = 0.f;
          }
        }
        if (!(ok = wait_warp(tail->dp_full[x & 1], x >> 1, abort_flag, a.dev_status))) break;
        tc_fence_after();
        float dp[64];
        tmem_ld32(dp_addr, dp);
        tmem_ld32(dp_addr + 32, dp + 32);
        tmem_wait_ld();
        pin<64>(dp);
        tc_fence_before();
        mbar_arrive(smem_u32(&tail->dp_free));
        const float2 nd = make_float2(neg_delta, neg_delta);
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          const float2 y = mul2(make_float2(w[j], w[j + 1]),
                                add2(make_float2(dp[j], dp[j + 1]), nd));
          dp[j] = y.x;
          dp[j + 1] = y.y;
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
        mbar_arrive(smem_u32(&tail->dz_full[x & 1]));
      }
      if (!ok) break;
      more = take(item + 1);
      if (count > 0) {
        if (!(ok = wait_warp(tail->done, used, abort_flag, a.dev_status))) break;
        ++used;
        tc_fence_after();
      }
      // dq, half of the columns in each warpgroup
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.dq) + b * a.sdq[0] + h * a.sdq[2];
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
        store_rows32(out, a.sdq[1], row - lane, a.Sq, c, a.D, o, a.scale);
      }
      tc_fence_before();  // dq has been read before the next item's dz is announced
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
  static constexpr uint32_t kTailBytes = 3072;  // as for dq
  static constexpr uint32_t kBytes = kTailBytes + (2 + kQSlots + kESlots) * kTileBytes;
  static constexpr uint32_t kAsked = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
};
struct DkvTail {
  float sub[2][kTile], neg_delta[2][kTile];  // of a step's queries, copied with dO
  uint64_t k_full, q_full[3], e_full[2];
  uint64_t s_full, p_full, dz_full, done, drain;
  uint64_t dp_full[2];  // by step modulo 2: two may be done before the copying thread looks
  uint32_t tmem;
  int abort_flag, lo, hi;
  int same[2], equal;  // query tiles that share the keys' one document: first, end, count
};
// Where the blocks of a cluster add up (over the tiles): fp32 rows of dk, then
// of dv, from every rank.
template <int DH>
constexpr int kJoinPitch = DH + 4;


template <int DH, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) k_attn_dkv(const __grid_constant__ Params p) {
  using L = DkvLayout<DH>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t *smem = raw + L::kTailBytes;
  DkvTail *tail = reinterpret_cast<DkvTail *>(raw);
  static_assert(sizeof(DkvTail) <= L::kTailBytes, "tail");
  const AttnArgs &a = p.a;
  if ((smem_u32(raw) & 1023) != 0) {  // not met: the tiles' layout needs it
    if (threadIdx.x == 0) atomicOr(a.dev_status, kDevErrTimeout);
    return;  // (the same in every block: none waits for another)
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  // the first keys of a causal mask are seen by most queries: first; with
  // documents in the order of falling work that was found with their ranges
  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int ranks = p.cluster, rank = static_cast<int>(blockIdx.x) % ranks;
  const int item = static_cast<int>(blockIdx.x) / ranks, g = item % a.Hk;
  // The dq kernel before this one writes nothing that is read here, and lets
  // it start only when what came before dq has finished: no wait, so that
  // blocks begin on the SMs that dq leaves first.  They wait before they
  // leave instead: this kernel ends after dq.  (Without queries there is no dq;
  // where dq forms delta of some row, the copying thread waits before it reads that.)
  if (a.Sq == 0) griddep_wait();
  griddep_launch_dependents();
  const int entry = a.order != nullptr ? __ldcg(a.order + item / a.Hk) : item / a.Hk;
  const int b = a.order != nullptr ? entry / ktiles : entry % a.B;
  const int kt = a.order != nullptr ? entry % ktiles : entry / a.B;
  const int key0 = kt * kTile, off = a.Sk - a.Sq;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->k_full), 1);
    for (int s = 0; s < L::kQSlots; ++s) mbar_init(smem_u32(&tail->q_full[s]), 1);
    for (int s = 0; s < L::kESlots; ++s) mbar_init(smem_u32(&tail->e_full[s]), 1);
    mbar_init(smem_u32(&tail->s_full), 1);
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&tail->dp_full[s]), 1);
    mbar_init(smem_u32(&tail->p_full), kPairThreads);
    mbar_init(smem_u32(&tail->dz_full), kPairThreads);
    mbar_init(smem_u32(&tail->done), 1);
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
    tail->lo = tail->same[0] = INT_MAX;
    tail->hi = tail->same[1] = tail->equal = 0;
    fence_barrier_init();
    tma_prefetch(&p.m.q);
    tma_prefetch(&p.m.k);
    tma_prefetch(&p.m.v);
    tma_prefetch(&p.m.d_o);
  }
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
  if (a.q_docs != nullptr) {
    const DocRange kr = doc_range(a.k_ranges, int64_t(b) * ktiles + kt);
    for (int n = first + threadIdx.x; n < qtiles; n += kThreads) {
      const DocRange qr = doc_range(a.q_ranges, int64_t(b) * qtiles + n);
      if (docs_meet(kr, qr)) {
        atomicMin(&tail->lo, n);
        atomicMax(&tail->hi, n + 1);
      }
      if (docs_equal(kr, qr)) {
        atomicMin(&tail->same[0], n);
        atomicMax(&tail->same[1], n + 1);
        atomicAdd(&tail->equal, 1);
      }
    }
  } else if (threadIdx.x == 0) {
    tail->lo = first;
    tail->hi = tail->same[1] = tail->equal = qtiles;
    tail->same[0] = 0;
  }
  __syncthreads();
  const int end = uniform(tail->hi), begin = uniform(min(tail->lo, end));
  const int per_head = end - begin, all = per_head * a.group;
  // Queries that see the keys of one tile only have delta from dq: with
  // documents any may, else those that see the first key tile alone.  Where
  // these all lie in the first of a head's query tiles, its step comes last.
  const bool from_dq =
      a.q_docs != nullptr || (kt == 0 && (a.causal ? off < kTile : a.Sk <= kTile));
  const int turn =
      from_dq && a.q_docs == nullptr && a.causal && off >= 0 && per_head > 1 ? 1 : 0;
  auto tile_at = [&](int place) {
    place += turn;
    return begin + (place < per_head ? place : place - per_head);
  };
  // step i of the item: query head g * group + i / per_head, tile tile_at(i %
  // per_head); this rank's are `count` from step0 on
  const int step0 = static_cast<int>(int64_t(all) * rank / ranks);
  const int count = static_cast<int>(int64_t(all) * (rank + 1) / ranks) - step0;

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
               tile_at((step0 + i) % per_head) * kTile,
               g * a.group + (step0 + i) / per_head);
          ++nq;
        };
        load_q(0);
        for (int i = 0; i < count; ++i) {
          // dP of step i - 1 is done, hence everything of step i - 2: the slots
          // of Q's tile i - 2 and dO's.  (dP of step i + 1, the next on its
          // barrier, needs the copy that is asked for after this wait: the phase
          // waited for is the barrier's open one or the one before.)
          if (i >= L::kESlots &&
              !mbar_wait(smem_u32(&tail->dp_full[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort_flag,
                         a.dev_status))
            break;
          const int s = i % L::kESlots, tile = tile_at((step0 + i) % per_head);
          if (from_dq && (turn == 0 || tile == begin)) griddep_wait();
          mbar_expect_tx(smem_u32(&tail->e_full[s]), L::kTileBytes + 2 * kTile * 4);
          const int64_t stat =
              ((static_cast<int64_t>(b) * a.Hq + g * a.group + (step0 + i) / per_head) * qtiles +
               tile) * kTile;
          bulk_load(smem_u32(tail->sub[s]), a.sub + stat, kTile * 4, smem_u32(&tail->e_full[s]));
          bulk_load(smem_u32(tail->neg_delta[s]), a.neg_delta + stat, kTile * 4,
                    smem_u32(&tail->e_full[s]));
          load(e_ring + s * L::kTileBytes, &p.m.d_o, tail->e_full[s], tile * kTile,
               g * a.group + (step0 + i) / per_head);
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
        return a.q_docs != nullptr && i < count
                   ? doc_range(a.q_ranges, int64_t(b) * qtiles + tile_at((step0 + i) % per_head)).padded
                   : 0;
      };
      int pads_q = padded(0), pads_e = pads_q;
      // a tile of step i has landed; without the rows of padding
      auto clear = [&](int now, int tile, int i) {
        const int token = tile_at((step0 + i) % per_head) * kTile;
        if (now != 0)
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
        commit(on, smem_u32(&tail->dp_full[i & 1]));
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
    if (ranks > 1) {  // the pairs' two barriers of the cluster
      __syncwarp();
      cluster_sync();
      cluster_sync();
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
    bool ok = true;
    // query tiles of the keys' one document, where they lie in one run
    const int same0 = tail->same[0];
    const int same1 = tail->equal == tail->same[1] - same0 ? tail->same[1] : same0;
    int head = g * a.group, place = 0;  // of this step
    if (count > 0) {
      head += step0 / per_head;
      place = step0 % per_head;
    }
    for (int i = 0; i < count; ++i) {
      const int n = tile_at(place), q0 = n * kTile + half * 64;
      const ScoreConst sc = score_const(a, head, true);
      const bool same = n >= same0 && n < same1;
      const bool whole = same && n * kTile >= all_from;
      int qd[2];
      if (!same) load_docs(a.q_docs + b * a.qds + q0, a.Sq - q0, qd);
      // the step's scores, and its statistics
      if (!(ok = wait_warp(tail->s_full, i, abort_flag, a.dev_status) &&
                 wait_warp(tail->e_full[i % L::kESlots], i / L::kESlots, abort_flag, a.dev_status)))
        break;
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
        if (!same) same_doc(kd, qd, keep);
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
      if (!(ok = wait_warp(tail->dp_full[i & 1], i >> 1, abort_flag, a.dev_status))) break;
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
      if (++place == per_head) {
        place = 0;
        ++head;
      }
    }
    if (ok && count > 0) {
      ok = wait_warp(tail->done, 0, abort_flag, a.dev_status);
    }
    ok = !named_bar_red_or(1, kPairThreads, !ok);
    // one warpgroup has dk, the other dv
    const uint32_t sum_addr = tmem + lanes + (half == 0 ? 384 : 256);
    const int64_t *stride = half == 0 ? a.sdk : a.sdv;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(half == 0 ? a.dk : a.dv) + b * stride[0] +
                         g * stride[2];
    const float by = half == 0 ? a.scale : 1.f;
    auto sum_of = [&](int c, float (&o)[32]) {
      if (count > 0) {
        tmem_ld32(sum_addr + c, o);
        tmem_wait_ld();
        pin<32>(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
      }
    };
    tc_fence_after();
    if (ranks == 1) {
      if (ok)
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          float o[32];
          sum_of(c, o);
          store_rows32(out, stride[1], key - lane, a.Sk, c, a.D, o, by);
        }
    } else {
      cluster_sync();  // every block is done with the tiles that the sums go over
      const int rows = kTile / ranks;  // of each rank
      constexpr int kPitch = kJoinPitch<DH>;
      float *join = reinterpret_cast<float *>(smem) + half * kTile * kPitch;
      const uint32_t to = dsmem_map(
          smem_u32(join + (rank * rows + r % rows) * kPitch), static_cast<uint32_t>(r / rows));
#pragma unroll 1
      for (int c = 0; c < DH; c += 32) {
        float o[32];
        sum_of(c, o);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          dsmem_st_f4(to + (c + e) * 4, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
      }
      cluster_sync();
      // this rank's rows, the ranks' sums in order
      if (ok)
        for (int x = r; x < rows * (DH / 4); x += kTile) {
          const int lr = x / (DH / 4), c = x % (DH / 4) * 4, at = key0 + rank * rows + lr;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int s = 0; s < ranks; ++s) {
            const float4 v =
                *reinterpret_cast<const float4 *>(join + (s * rows + lr) * kPitch + c);
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
          }
          if (at < a.Sk && c < a.D)
            *reinterpret_cast<uint2 *>(out + at * stride[1] + c) =
                make_uint2(pack_bf16(acc.x * by, acc.y * by), pack_bf16(acc.z * by, acc.w * by));
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  griddep_wait();
}

template <int DH, bool CAP, bool BIAS>
cudaError_t start_dq(const Params &p, int sms, cudaStream_t s) {
  constexpr size_t smem = DqLayout<DH>::kAsked;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_attn_dq<DH, CAP, BIAS>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_attn_dq<DH, CAP, BIAS>, dim3(p.items < sms ? p.items : sms), dim3(kThreads),
                    smem, s, p);
}
template <int DH, bool CAP, bool BIAS>
cudaError_t start_dkv(const Params &p, int, cudaStream_t s) {
  constexpr size_t smem = DkvLayout<DH>::kAsked;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(k_attn_dkv<DH, CAP, BIAS>, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.items) * p.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_attn_dkv<DH, CAP, BIAS>, p);
}

}  // namespace

#define LORA_ATTN_VARIANT(f)                                                            \
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;                             \
  if (a.D <= 64)                                                                        \
    return cap ? (bias ? f<64, true, true>(p, sms, s) : f<64, true, false>(p, sms, s))  \
               : (bias ? f<64, false, true>(p, sms, s) : f<64, false, false>(p, sms, s)); \
  return cap ? (bias ? f<128, true, true>(p, sms, s) : f<128, true, false>(p, sms, s))  \
             : (bias ? f<128, false, true>(p, sms, s) : f<128, false, false>(p, sms, s))

cudaError_t launch_attn_stats(const AttnArgs &a, cudaStream_t s) {
  const int64_t blocks = int64_t(a.B) * ((a.Sq + kTile - 1) / kTile * (kTile / 32)) *
                         ((a.Hq + kStatWarps - 1) / kStatWarps);
  return launch_pdl(a.D <= 64 ? k_attn_stats<64> : k_attn_stats<128>,
                    dim3(static_cast<unsigned>(blocks)), dim3(32 * kStatWarps), 0, s, a);
}

cudaError_t launch_attn_dq(const AttnArgs &a, const AttnBwdMaps &m, int sms, cudaStream_t s) {
  const Params p{a, m, a.B * a.Hq * ((a.Sq + kTile - 1) / kTile), 1};
  LORA_ATTN_VARIANT(start_dq);
}

cudaError_t launch_attn_dkv(const AttnArgs &a, const AttnBwdMaps &m, int sms, cudaStream_t s) {
  Params p{a, m, a.B * a.Hk * ((a.Sk + kTile - 1) / kTile), 1};
  // Blocks of an item: while a cluster of twice as many fits the SMs at once,
  // or, where the items differ in work, would leave each at least 16 steps (of
  // some 1.5 us; a block's beginning and end, and the meeting of the cluster,
  // take some 12 us).  Items, steps, and backward by blocks of an item, 1 / 2 /
  // 4 / 8: causal 128, 64: 144 / 117 / 146 / 220 us; 64, 128: 220 / 142 / 113 /
  // 158; 128, 16: 62 / 72 / 97 / 165; without a mask 128, 64: 182 / 197 / 219 / 281.
  const int steps = a.group * ((a.Sq + kTile - 1) / kTile);
  while (p.cluster < 8 && steps >= 4 * p.cluster &&
         (p.items * p.cluster * 2 <= sms ||
          ((a.causal || a.q_docs != nullptr) && p.items * p.cluster < sms &&
           steps >= 32 * p.cluster)))
    p.cluster *= 2;
  LORA_ATTN_VARIANT(start_dkv);
}

}  // namespace lora
