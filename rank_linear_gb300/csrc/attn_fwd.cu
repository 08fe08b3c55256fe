// attn_fwd.cu -- attention forward on the tensor cores (include/lora_attention.h).
//
// An item is 256 queries of one head, as two tiles of 128, and one pass over
// the keys in tiles of 128: S = Q K^T into TMEM, softmax in registers (a
// thread owns a whole row: no shuffles), P back into TMEM as bf16 over S, and
// O += P V with P as the TMEM operand.  While the softmax of one tile runs,
// the tensor core works for the other.  The running maximum is only followed
// when it has moved by more than 2^8: until then P is relative to the old one
// (at most 256, exact in fp32 sums and no worse rounded to bf16), so that O
// in TMEM is hardly ever rescaled.  P is rounded to bf16 because the tensor
// core multiplies it with bf16 V: o is then 0.0019 to 0.0024 of its norm from
// 64 bits where rounding it alone takes 0.0017; two bf16 parts of P, as with
// one token, would be a product more for every two.
//
// Blocks stay (one per SM) and take item after item, so that an item's copies
// and first scores run while the one before it is written out.  A scheduling
// warp hands items out: in order of falling work without documents, from a
// counter with them (their work varies).  Where the last round would leave
// SMs without an item, its items are cut along the keys (see attn_fwd_plan):
// 2048 queries over 16000 keys 329 -> 307 us, 50 over 30000 with 4 heads 277 ->
// 31 us.  Few queries share an item with the heads of their group, which read
// the same keys: 16 over 8192, four times 32 heads over 8, 85 -> 44 us (K and V
// alone take 20: the parts meet in memory, and an item has 64 rows of 256).
//
// TMEM: S/P of the two tiles at columns 0 and 128, O at 256 and 384.
//
// Measured (32 heads of 128, 8 key heads): 8192 x 8192 without a mask 623 us
// (1765 TFLOP/s, 0.90 of what a large bf16 product reaches), causal 334 us
// (1645), heads of 64 causal 292 us (940: the exponentials take as long as the
// products), 4096 causal 97 us (1415); with capped scores 168 us, 244 us where
// many are beyond the cap, with a distance bias 134 us (one or two more
// operations a pair); five documents in 8192 139 us.  Bound by the
// tensor cores where a block has many steps; an item begins and ends in some
// 4 us that overlap its neighbours' steps only in part, and 256-row items
// leave work unused along the diagonal and at documents' edges.
#include "attn.cuh"
#include "host.h"

namespace lora {
namespace {

// Two softmax warpgroups, and one whose warps issue the copies, the MMAs and
// the items.  168 registers a thread at launch; the softmax threads, which
// hold a row of scores, take 224 and leave the others 56 (2 * 224 + 56 = 3 * 168).
constexpr int kThreads = 384, kSoftmaxRegs = 224, kIssueRegs = 56;
constexpr float kRescaleAt = 8.f;
constexpr int kItemSlots = 2, kItemReaders = 10;  // warps that read an item

template <int DH>
struct Layout {
  static constexpr uint32_t kTileBytes = kTile * DH * 2;
  // rings of K and V tiles; a V tile is asked for first and given back last
  static constexpr int kKSlots = DH == 64 ? 4 : 2, kVSlots = kKSlots + 1;
  static constexpr uint32_t kBytes = (2 + kKSlots + kVSlots) * kTileBytes;
};

// 256 queries from row0 of head h, batch entry b, and the key tiles [lo, hi)
// that some row of each of the two tiles sees; [begin, begin + count) covers
// both.  count < 0: no more items.
struct Item {
  int row0, h, b, lo[2], hi[2], begin, count;
  int same[2][2];  // key tiles [0], ..., [1] - 1 of the query tile's one document
};

struct Tail {
  uint64_t q_full, q_free, k_full[4], v_full[5];
  uint64_t passed[5];  // the products before step x (over all items), at x modulo kVSlots
  uint64_t s_full[2], p_full[2][2], o_done[2], drain;
  uint64_t item_full[kItemSlots], item_free[kItemSlots];
  Item item[kItemSlots];
  uint32_t tmem;
  int abort_flag;
};

struct Params {
  AttnArgs a;
  AttnMaps m;
  int items;
  AttnFwdPlan t;
  float2 *stat;
  float4 *part;
};

// The first worker that has part of item i, and the last (see AttnFwdPlan:
// worker j's share is [j tail / workers, (j + 1) tail / workers) of the items).
__device__ __forceinline__ int first_worker(const AttnFwdPlan &t, int i) {
  return i * t.workers / t.tail;
}
__device__ __forceinline__ int last_worker(const AttnFwdPlan &t, int i) {
  return ((i + 1) * t.workers - 1) / t.tail;
}

// The result of the block's item n has this place among the parts of cut
// items; -1: it is a whole item's.
__device__ __forceinline__ int part_of(const AttnFwdPlan &t, int n) {
  if (n < t.rounds) return -1;
  const int place = blockIdx.x, i = place * t.tail / t.workers + n - t.rounds;
  return i * t.segments + place - first_worker(t, i);
}

// Reads item n of the block: false where there is none (or on an abort).
__device__ __forceinline__ bool next_item(Tail *tail, int n, Item &item, volatile int *abort_flag,
                                          unsigned *dev_status) {
  const int s = n % kItemSlots;
  if (!wait_warp(tail->item_full[s], n / kItemSlots, abort_flag, dev_status)) return false;
  item = tail->item[s];
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(smem_u32(&tail->item_free[s]));
  return item.count >= 0;
}

// SPECIAL: items of the last round are cut along the keys, or rows are heads of
// a group side by side (a variant: in the same kernel it costs the softmax
// registers, and packed documents 4 %).
template <int DH, bool CAP, bool BIAS, bool SPECIAL>
__global__ void __launch_bounds__(kThreads, 1) k_attn_fwd(const __grid_constant__ Params p) {
  using L = Layout<DH>;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Tail *tail = reinterpret_cast<Tail *>(smem + L::kBytes);
  const AttnArgs &a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort_flag = &tail->abort_flag;

  const int off = a.Sk - a.Sq;
  const int ktiles = (a.Sk + kTile - 1) / kTile, qtiles = (a.Sq + kTile - 1) / kTile;
  // rows: queries, or 2^shift heads of each
  const int shift = SPECIAL ? p.t.shift : 0, rows = a.Sq << shift;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&tail->q_full), 1);
    mbar_init(smem_u32(&tail->q_free), 1);
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
    for (int s = 0; s < kItemSlots; ++s) {
      mbar_init(smem_u32(&tail->item_full[s]), 1);
      mbar_init(smem_u32(&tail->item_free[s]), kItemReaders);
    }
    mbar_init(smem_u32(&tail->drain), 1);
    tail->abort_flag = 0;
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

  if (warp >= 8) {
    set_max_regs_down<kIssueRegs>();
    const uint32_t q_tile = smem_u32(smem), k_ring = q_tile + 2 * L::kTileBytes;
    const uint32_t v_ring = k_ring + L::kKSlots * L::kTileBytes;
    if (warp == 10) {
      // ------------------------------------------------------ items
      const int sets = a.Hq >> shift, heads = a.B * sets, blocks_q = p.items / heads;
      for (int n = 0;; ++n) {
        const int s = n % kItemSlots;
        if (n >= kItemSlots &&
            !wait_warp(tail->item_free[s], n / kItemSlots - 1, abort_flag, a.dev_status))
          break;
        // to and fro over the blocks, so that their sums of falling work match
        const int blocks = gridDim.x, place = blockIdx.x;
        int id = n * blocks + (n & 1 ? blocks - 1 - place : place);
        if (a.counter != nullptr && n > 0) {  // the first of each block is its own
          if (lane == 0) id = blocks + static_cast<int>(atomicAdd(a.counter, 1u));
          id = __shfl_sync(~0u, id, 0);
        }
        int from_part = 0, to_part = 1, parts = 0;
        if (SPECIAL && n >= p.t.rounds) {  // this block's share of the items that are cut
          const int i = place * p.t.tail / p.t.workers + n - p.t.rounds;
          parts = p.t.workers;
          from_part = max(place * p.t.tail - i * parts, 0);
          to_part = min((place + 1) * p.t.tail - i * parts, parts);
          id = place < parts && from_part < to_part ? p.t.rounds * blocks + i : p.items;
        }
        Item it = {};
        it.count = -1;
        if (id < p.items) {
          // the last queries, which see most keys of a causal mask, first
          const int qb = blocks_q - 1 - id / heads, bh = id % heads;
          it.b = bh / sets;
          it.h = bh % sets << shift;
          it.row0 = qb * kAttnQueries;
          const int prefix = a.prefix != nullptr ? a.prefix[it.b] : 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int first = it.row0 + t * kTile, last = (min(first + kTile, rows) - 1) >> shift;
            int lo = 0;
            int hi = first < rows ? max(0, (last_key(a, last + off, prefix) + kTile) / kTile) : 0;
            it.same[t][0] = 0;
            it.same[t][1] = INT_MAX;  // no documents: one
            if (a.q_docs != nullptr && hi > 0)
              doc_tiles(doc_range(a.q_ranges, int64_t(it.b) * qtiles + (first >> shift) / kTile),
                        a.k_ranges + int64_t(it.b) * ktiles, lo, hi, it.same[t]);
            it.lo[t] = lo;
            it.hi[t] = hi;
          }
          // the tiles either passes over
          const bool none0 = it.hi[0] == it.lo[0], none1 = it.hi[1] == it.lo[1];
          it.begin = none0 ? it.lo[1] : none1 ? it.lo[0] : min(it.lo[0], it.lo[1]);
          it.count = (none0 ? it.hi[1] : none1 ? it.hi[0] : max(it.hi[0], it.hi[1])) - it.begin;
          if (SPECIAL && parts > 0) {
            const int lo = it.begin + it.count * from_part / parts;
            const int hi = it.begin + it.count * to_part / parts;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              it.lo[t] = max(it.lo[t], lo);
              it.hi[t] = max(min(it.hi[t], hi), it.lo[t]);
            }
            // (a tile of the range that neither sees, between the two, is passed over)
            it.begin = lo;
            it.count = hi - lo;
          }
        }
        if (lane == 0) {
          tail->item[s] = it;
          mbar_arrive(smem_u32(&tail->item_full[s]));  // releases the item's words
          if (it.count > 0)  // what it begins with, towards L2
            for (int c = 0; c < DH; c += 64) {
              if (!SPECIAL) {
                tma_prefetch_4d(&p.m.q, c, it.row0, it.h, it.b);
                tma_prefetch_4d(&p.m.q, c, it.row0 + kTile, it.h, it.b);
              }
              tma_prefetch_4d(&p.m.k, c, it.begin * kTile, it.h / a.group, it.b);
              tma_prefetch_4d(&p.m.v, c, it.begin * kTile, it.h / a.group, it.b);
            }
        }
        __syncwarp();
        if (it.count < 0) break;
      }
    } else if (warp == 8) {
      // ------------------------------------------------------ TMA
      int x = 0, used = 0;  // tiles loaded so far, items with tiles
      bool ok = true;
      Item it;
      for (int n = 0; ok && next_item(tail, n, it, abort_flag, a.dev_status); ++n) {
        if (it.count == 0) continue;
        if (used > 0) ok = wait_warp(tail->q_free, used - 1, abort_flag, a.dev_status);
        if (!ok) break;
        const int g = it.h / a.group;
        auto load = [&](uint32_t dst, const CUtensorMap *tm, uint64_t &bar, int token, int head) {
          for (int c = 0; c < DH / 64; ++c)
            tma_load_4d(dst + c * kTile * 128, tm, smem_u32(&bar), c * 64, token, head, it.b);
        };
        if (lane == 0) {
          mbar_expect_tx(smem_u32(&tail->q_full), 2 * L::kTileBytes);
          for (int t = 0; t < 2; ++t)  // a second tile past the end reads as zeros
            if constexpr (SPECIAL)
              for (int c = 0; c < DH / 64; ++c)
                tma_load_5d(q_tile + t * L::kTileBytes + c * kTile * 128, &p.m.q,
                            smem_u32(&tail->q_full), c * 64, (it.row0 + t * kTile) >> shift,
                            it.h >> shift, it.b);
            else
              load(q_tile + t * L::kTileBytes, &p.m.q, tail->q_full, it.row0 + t * kTile, it.h);
        }
        ++used;
        for (int i = 0; i < it.count; ++i, ++x) {
          // K's slot is scored, and V's is read, before step x - kKSlots
          const int gone = x - L::kKSlots;
          if (gone >= 0 && !(ok = wait_warp(tail->passed[gone % L::kVSlots], gone / L::kVSlots,
                                            abort_flag, a.dev_status)))
            break;
          if (lane == 0) {
            const int ks = x % L::kKSlots, vs = x % L::kVSlots, token = (it.begin + i) * kTile;
            mbar_expect_tx(smem_u32(&tail->k_full[ks]), L::kTileBytes);
            load(k_ring + ks * L::kTileBytes, &p.m.k, tail->k_full[ks], token, g);
            mbar_expect_tx(smem_u32(&tail->v_full[vs]), L::kTileBytes);
            load(v_ring + vs * L::kTileBytes, &p.m.v, tail->v_full[vs], token, g);
          }
          __syncwarp();
        }
      }
      // copies in flight land before the CTA leaves
      if (lane == 0) {
        if (used > 0) mbar_wait_drain(smem_u32(&tail->q_full), (used - 1) & 1);
        for (int s = 0; s < L::kKSlots && s < x; ++s)
          mbar_wait_drain(smem_u32(&tail->k_full[s]), ((x - 1 - s) / L::kKSlots) & 1);
        for (int s = 0; s < L::kVSlots && s < x; ++s)
          mbar_wait_drain(smem_u32(&tail->v_full[s]), ((x - 1 - s) / L::kVSlots) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------ MMA
      // (a commit holds the queue of MMAs for some 90 cycles: as few as will do)
      const uint32_t on = elect_one();
      auto wait = [&](const uint64_t &bar, int phase) {
        return wait_warp(bar, phase, abort_flag, a.dev_status);
      };
      const auto p_cols = [](int kk) { return kk * 8; };
      int base = 0, used = 0;  // tiles and items with tiles before this item
      int turn[2] = {0, 0};    // score tiles done of each query tile
      bool ok = true;
      Item it;
      for (int n = 0; ok && next_item(tail, n, it, abort_flag, a.dev_status); ++n) {
        const int count = uniform(it.count), begin = uniform(it.begin), b = uniform(it.b);
        if (count == 0) continue;
        const int lo[2] = {uniform(it.lo[0]), uniform(it.lo[1])};
        const int hi[2] = {uniform(it.hi[0]), uniform(it.hi[1])};
        auto wait_k = [&](int i) {
          const int x = base + i;
          return wait(tail->k_full[x % L::kKSlots], x / L::kKSlots);
        };
        auto scores = [&](int t, int i) {
          mma_over_head<DH>(on, tmem + t * kTile, q_tile + t * L::kTileBytes,
                            k_ring + ((base + i) % L::kKSlots) * L::kTileBytes);
          commit(on, smem_u32(&tail->s_full[t]));
        };
        auto padded = [&](int i) {
          return a.q_docs != nullptr && i < count
                     ? doc_range(a.k_ranges, int64_t(b) * ktiles + begin + i).padded
                     : 0;
        };
        // V's tile i has landed; without the rows of padding
        int pads = padded(0);  // looked at a step later: not waited for here
        auto wait_v = [&](int i) {
          const int s = (base + i) % L::kVSlots, token = (begin + i) * kTile;
          if (!wait(tail->v_full[s], (base + i) / L::kVSlots)) return false;
          if (pads != 0)
            zero_padding_rows<DH>(smem + (2 + L::kKSlots + s) * L::kTileBytes,
                                  a.k_docs + b * a.kds + token, a.Sk - token);
          pads = padded(i + 1);
          return true;
        };
        if (!(ok = wait(tail->q_full, used) && wait_k(0))) break;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (begin >= lo[t] && begin < hi[t]) scores(t, 0);
        commit(on, smem_u32(&tail->passed[base % L::kVSlots]));
        if (count == 1) commit(on, smem_u32(&tail->q_free));
        if (!(ok = wait_v(0))) break;
        bool first[2] = {true, true};
        for (int i = 0; i < count && ok; ++i) {
          const int tile = begin + i;
          const bool more = i + 1 < count;
          const uint32_t vt = v_ring + ((base + i) % L::kVSlots) * L::kTileBytes;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (tile >= lo[t] && tile < hi[t]) {
              const uint32_t o = tmem + 256 + t * kTile, w = tmem + t * kTile;
              if (!(ok = wait(tail->p_full[t][0], turn[t]))) break;
              tc_fence_after();
              mma_over_tokens<DH, 0, 4>(on, o, w, p_cols, vt, !first[t]);
              if (!(ok = wait(tail->p_full[t][1], turn[t]))) break;
              tc_fence_after();
              mma_over_tokens<DH, 4, 8>(on, o, w, p_cols, vt, true);
              if (tile + 1 == hi[t]) commit(on, smem_u32(&tail->o_done[t]));
              first[t] = false;
              ++turn[t];
            }
            // While the queue is full: the steps before are given back, and the
            // waits for what the next step reads.
            if (t == 0) {
              if (i > 0) commit(on, smem_u32(&tail->passed[(base + i) % L::kVSlots]));
              if (more && !(ok = wait_k(i + 1))) break;
            } else if (more) {
              if (!(ok = wait_v(i + 1))) break;
            }
            tc_fence_after();
            if (tile + 1 >= lo[t] && tile + 1 < hi[t]) scores(t, i + 1);
          }
          if (i + 2 == count) commit(on, smem_u32(&tail->q_free));  // Q has been read
        }
        base += count;
        ++used;
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
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * kTile, o_addr = tmem + lanes + 256 + t * kTile;
    int turn = 0, done = 0;  // score tiles, and items with tiles, of this query tile
    bool ok = true;
    Item it;
    for (int item = 0; ok && next_item(tail, item, it, abort_flag, a.dev_status); ++item) {
      const int b = it.b, first = it.row0 + t * kTile;
      if (first >= rows) continue;
      const int lo = it.lo[t], hi = it.hi[t], row = first + (threadIdx.x & 127);
      const int query = row >> shift, h = it.h + (row & ((1 << shift) - 1));
      const int prefix = a.prefix != nullptr ? a.prefix[b] : 0;
      const ScoreConst sc = score_const(a, h);
      const int pos = query + off;
      const int last = row < rows ? last_key(a, pos, prefix) : -1;
      const int first_last = last_key(a, (first >> shift) + off, prefix);  // of the first row
      const int same0 = it.same[t][0], same1 = it.same[t][1];
      int qd = -1;
      if (a.q_docs != nullptr && row < rows) qd = a.q_docs[b * a.qds + query];
      float m = -INFINITY;  // the maximum that P is relative to, in log2 units
      float2 l2 = make_float2(0.f, 0.f);
      for (int n = lo; n < hi; ++n, ++turn) {
        // does the mask leave the whole tile?
        const bool same = n >= same0 && n < same1;
        const bool whole = same && n * kTile + kTile - 1 <= first_last;
        int kd[4];
        if (!same) load_docs(a.k_docs + b * a.kds + n * kTile, a.Sk - n * kTile, kd);
        if (!(ok = wait_warp(tail->s_full[t], turn, abort_flag, a.dev_status))) break;
        tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, s + c * 32);
        tmem_wait_ld();
        pin<kTile>(s);
        if constexpr (CAP || BIAS) {
          const float d0 = static_cast<float>(pos - n * kTile);
          auto transform = [&](bool small) {
#pragma unroll
            for (int j = 0; j < kTile; j += 2) {
              const float2 x =
                  scores2<CAP, BIAS>(sc, make_float2(s[j], s[j + 1]), d0 - j, -1.f, small);
              s[j] = x.x;
              s[j + 1] = x.y;
            }
          };
          if (!CAP || all_small<kTile>(sc, s))
            transform(true);
          else
            transform(false);
        }
        if (!whole) {
          uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
          if (!same) same_doc(qd, kd, keep);
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
      if (!ok) break;
      if (lo < hi) {
        if (!(ok = wait_warp(tail->o_done[t], done, abort_flag, a.dev_status))) break;
        ++done;
        tc_fence_after();
      }
      const float l = l2.x + l2.y;
      const int part = SPECIAL ? part_of(p.t, item) : -1;
      if (part >= 0) {  // part of an item: joined with the others later
        const int r = threadIdx.x & 127;
        p.stat[static_cast<int64_t>(part) * kAttnQueries + t * kTile + r] = make_float2(m, l);
        float4 *to =
            p.part + static_cast<int64_t>(part) * (DH / 4) * kAttnQueries + t * kTile + r;
        if (lo < hi)
#pragma unroll 1
          for (int c = 0; c < DH; c += 32) {
            float o[32];
            tmem_ld32(o_addr + c, o);
            tmem_wait_ld();
            pin<32>(o);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              to[(c + e) / 4 * kAttnQueries] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        tc_fence_before();
        continue;
      }
      // straight to global memory: Q's shared memory is already the next item's
      const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: nothing was seen (NaN stays NaN)
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.o) + b * a.so[0] +
                           (SPECIAL ? h & ~((1 << shift) - 1) : h) * a.so[2];
#pragma unroll 1
      for (int c = 0; c < DH; c += 32) {
        float o[32];
        if (lo < hi) {
          tmem_ld32(o_addr + c, o);
          tmem_wait_ld();
          pin<32>(o);
        }
        if (l == 0.f)
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        store_rows32(out, a.so[1], row - lane, rows, c, a.D, o, inv, shift, SPECIAL ? a.so[2] : 0);
      }
      tc_fence_before();  // O has been read before the next item's P is announced
      if (a.lse != nullptr && row < rows)
        a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Sq + query] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that were cut, in the order of the keys: 32
// queries x 32 elements of the head a block, a thread four elements of a query.
constexpr int kJoinWarps = 8;
template <int DH>
__global__ void __launch_bounds__(32 * kJoinWarps) k_attn_fwd_join(const __grid_constant__ Params p) {
  __shared__ float tile[32][33];
  const AttnArgs &a = p.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  constexpr int kRows = kAttnQueries / 32, kCols = DH / 32;
  const int i = blockIdx.x / (kRows * kCols), col = blockIdx.x / kRows % kCols * 32;
  const int r = blockIdx.x % kRows * 32 + lane;
  const int shift = p.t.shift, rows = a.Sq << shift, sets = a.Hq >> shift;
  const int heads = a.B * sets, blocks_q = p.items / heads, id = p.items - p.t.tail + i;
  const int row0 = (blocks_q - 1 - id / heads) * kAttnQueries, bh = id % heads;
  const int parts = last_worker(p.t, i) - first_worker(p.t, i) + 1;
  griddep_wait();
  griddep_launch_dependents();
  if (row0 + r - lane >= rows) return;
  const float2 *stat = p.stat + static_cast<int64_t>(i) * p.t.segments * kAttnQueries + r;
  const float4 *from = p.part +
                       (static_cast<int64_t>(i) * p.t.segments * (DH / 4) + col / 4 + warp) *
                           kAttnQueries + r;
  float m = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float2 x = __ldcg(stat + s * kAttnQueries);
    if (x.y != 0.f) m = fmaxf(m, x.x);
  }
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float2 x = __ldcg(stat + s * kAttnQueries);
    if (x.y != 0.f) {  // else nothing was seen, and there may be no output
      const float by = ex2(x.x - m);
      const float4 v = __ldcg(from + static_cast<int64_t>(s) * (DH / 4) * kAttnQueries);
      l = fmaf(by, x.y, l);
      o.x = fmaf(by, v.x, o.x);
      o.y = fmaf(by, v.y, o.y);
      o.z = fmaf(by, v.z, o.z);
      o.w = fmaf(by, v.w, o.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  tile[lane][warp * 4] = o.x * inv;
  tile[lane][warp * 4 + 1] = o.y * inv;
  tile[lane][warp * 4 + 2] = o.z * inv;
  tile[lane][warp * 4 + 3] = o.w * inv;
  const int b = bh / sets, h0 = bh % sets << shift, mask = (1 << shift) - 1;
  if (a.lse != nullptr && col == 0 && warp == 0 && row0 + r < rows)
    a.lse[(static_cast<int64_t>(b) * a.Hq + h0 + (r & mask)) * a.Sq + ((row0 + r) >> shift)] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  __syncthreads();
  // eight lanes to a row of 32 elements
  const int y = threadIdx.x / 8, c = threadIdx.x % 8 * 4, row = row0 + r - lane + y;
  if (row < rows && col + c < a.D) {
    const int64_t at = b * a.so[0] + static_cast<int64_t>(row >> shift) * a.so[1] +
                       (h0 + (row & mask)) * a.so[2];
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at + col + c) =
        make_uint2(pack_bf16(tile[y][c], tile[y][c + 1]), pack_bf16(tile[y][c + 2], tile[y][c + 3]));
  }
}

// Ranges of the documents of 128-token tiles of the queries, then of the keys,
// one warp per tile; zeroes the counters that items are handed out from.
__global__ void k_attn_ranges(const AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x < kAttnCounters) a.counter[threadIdx.x] = 0;
  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
  const bool keys = w >= a.B * qtiles;
  const int i = keys ? w - a.B * qtiles : w, tiles = keys ? ktiles : qtiles;
  if (i >= a.B * tiles) return;
  const int b = i / tiles, n = i % tiles, S = keys ? a.Sk : a.Sq;
  const int *docs = keys ? a.k_docs + b * a.kds : a.q_docs + b * a.qds;
  int lo = INT_MAX, hi = -1, padded = 0;
#pragma unroll
  for (int c = 0; c < kTile / 32; ++c) {
    const int at = n * kTile + 32 * c + lane;
    if (at < S) {
      const int d = docs[at];
      if (d < 0) {
        padded = 1;
      } else {
        lo = min(lo, d);
        hi = max(hi, d);
      }
    }
  }
  lo = __reduce_min_sync(~0u, lo);
  hi = __reduce_max_sync(~0u, hi);
  padded = __any_sync(~0u, padded);
  if (lane == 0) const_cast<int4 *>(keys ? a.k_ranges : a.q_ranges)[i] = make_int4(lo, hi, padded, 0);
}

// Key tiles in the order of falling work (the query tiles that see them), by
// one block: a counting sort into kBuckets.  The order inside a bucket may
// differ from run to run; no result depends on it.
constexpr int kOrderThreads = 1024, kBuckets = 1024;
__global__ void __launch_bounds__(kOrderThreads) k_attn_order(const AttnArgs a) {
  __shared__ int count[kBuckets];
  griddep_wait();
  griddep_launch_dependents();
  const int qtiles = (a.Sq + kTile - 1) / kTile, ktiles = (a.Sk + kTile - 1) / kTile;
  const int off = a.Sk - a.Sq, tiles = a.B * ktiles;
  count[threadIdx.x] = 0;
  __syncthreads();
  auto bucket = [&](int i) {  // 0: most work
    const int b = i / ktiles, n = i % ktiles;
    const DocRange kr = doc_range(a.k_ranges, i);
    const int prefix = a.prefix != nullptr ? a.prefix[b] : 0;
    const int first = a.causal && n * kTile >= prefix ? max(0, n * kTile - off) / kTile : 0;
    int from = INT_MAX, to = 0;
    for (int x = first; x < qtiles; ++x)
      if (docs_meet(kr, doc_range(a.q_ranges, int64_t(b) * qtiles + x))) {
        from = min(from, x);
        to = x + 1;
      }
    const int work = max(0, to - min(from, to));
    return kBuckets - 1 - static_cast<int>(int64_t(work) * (kBuckets - 1) / max(qtiles, 1));
  };
  // (a tile's bucket is found twice where a thread has more than one)
  const int mine = threadIdx.x < tiles ? bucket(threadIdx.x) : 0;
  if (threadIdx.x < tiles) atomicAdd(&count[mine], 1);
  for (int i = threadIdx.x + kOrderThreads; i < tiles; i += kOrderThreads)
    atomicAdd(&count[bucket(i)], 1);
  __syncthreads();
  // each bucket's first place
  const int own = count[threadIdx.x];
  int sum = own;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(~0u, sum, d);
    if (threadIdx.x % 32 >= d) sum += y;
  }
  __shared__ int warps[32];
  if (threadIdx.x % 32 == 31) warps[threadIdx.x / 32] = sum;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < static_cast<int>(threadIdx.x) / 32; ++w) before += warps[w];
  count[threadIdx.x] = before + sum - own;
  __syncthreads();
  int *order = const_cast<int *>(a.order);
  if (threadIdx.x < tiles) order[atomicAdd(&count[mine], 1)] = threadIdx.x;
  for (int i = threadIdx.x + kOrderThreads; i < tiles; i += kOrderThreads)
    order[atomicAdd(&count[bucket(i)], 1)] = i;
}

constexpr int kPlanSms = 152;  // of a GB300: the plan is one of sizes alone

template <int DH, bool CAP, bool BIAS, bool SPECIAL>
cudaError_t launch_as(const Params &p, int blocks, cudaStream_t s) {
  const size_t smem = Layout<DH>::kBytes + sizeof(Tail) + 1024;
  auto *kernel = k_attn_fwd<DH, CAP, BIAS, SPECIAL>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), smem, s, p);
}
template <int DH, bool CAP, bool BIAS>
cudaError_t launch(const Params &p, int sms, cudaStream_t s) {
  if (p.t.special()) {
    const int whole = p.items < kPlanSms ? p.items : kPlanSms;
    return launch_as<DH, CAP, BIAS, true>(p, p.t.rounds == 0 ? p.t.workers : whole, s);
  }
  return launch_as<DH, CAP, BIAS, false>(p, p.items < sms ? p.items : sms, s);
}

}  // namespace

cudaError_t launch_attn_ranges(const AttnArgs &a, cudaStream_t s) {
  const int64_t tiles = int64_t(a.B) * ((a.Sq + kTile - 1) / kTile + (a.Sk + kTile - 1) / kTile);
  return launch_pdl(k_attn_ranges, dim3(static_cast<unsigned>((tiles + 7) / 8)), dim3(256), 0, s, a);
}
cudaError_t launch_attn_order(const AttnArgs &a, cudaStream_t s) {
  return launch_pdl(k_attn_order, dim3(1), dim3(kOrderThreads), 0, s, a);
}

// Cuts the items of the last round, which fewer than all blocks would have,
// where that is worth it.  In steps (256 queries x 128 keys, 1.4 us): whole,
// they take as long as the longest; in shares, that times items / workers, and
// on top some 5 steps for the second item of a share and the join's launch,
// and for the parts' way out and back some 1 / 22 each (heads of 128;
// half that where only the first 128 of the queries are there).
// Measured, whole and cut, by what this makes of it (steps saved over their
// cost): 0.6: 33 and 35 us, 33 and 33; 1.0: 625 and 625; 1.1: 164 and 164; 1.2:
// 23 and 18, 53 and 45; 1.4: 31 and 23, 29 and 21; 2.1: 66 and 51; 6: 475 and 367.  No share of less than 4 steps, at most some 32 parts of an item.
// With documents the items' work is not known here: they are cut only where
// there is less than a round of them, else taken from a counter.
//
// Before that, where a group's heads fit an item together, as many as do share
// one: K and V are then read and multiplied once for them.
AttnFwdPlan attn_fwd_plan(int64_t B, int64_t Hq, int group, int64_t Sq, int64_t Sk, int D,
                          bool causal, bool prefix, bool docs) {
  AttnFwdPlan t;
  const int64_t queries = Sq;
  while (t.shift < 7 && group % (2 << t.shift) == 0 && 2 * Sq <= kAttnQueries) {
    ++t.shift;
    Sq *= 2;
  }
  const int64_t heads = B * (Hq >> t.shift), blocks_q = (Sq + kAttnQueries - 1) / kAttnQueries;
  const int64_t items = heads * blocks_q, rounds = items / kPlanSms;
  const int64_t tail = items - rounds * kPlanSms;
  if (tail == 0 || Sk == 0 || (docs && rounds > 0)) return t;
  int64_t keys = Sk;  // that the longest of the tail sees
  if (causal && !prefix) {
    const int64_t end = (blocks_q - rounds * kPlanSms / heads) * kAttnQueries;
    keys = ((end < Sq ? end : Sq) >> t.shift) + Sk - queries;
  }
  const int64_t steps = keys > 0 ? (keys + kTile - 1) / kTile : 0;
  int64_t workers = tail * steps / 4;
  if (workers > 32 * tail) workers = 32 * tail;
  if (workers > kPlanSms) workers = kPlanSms;
  if (workers <= tail) return t;
  const double saved = steps - double(steps) * tail / workers;
  const double part = (D <= 64 ? 0.5 : 1.0) * (Sq <= kTile ? 0.5 : 1.0) / 22;
  const double cost = 5 + part * (tail + workers);
  if (saved < 1.1 * cost) return t;
  t.rounds = static_cast<int>(rounds);
  t.tail = static_cast<int>(tail);
  t.workers = static_cast<int>(workers);
  t.segments = static_cast<int>((workers + tail - 1) / tail + 1);
  return t;
}
static int items_of(const AttnArgs &a, const AttnFwdPlan &t) {
  return a.B * (a.Hq >> t.shift) * (((a.Sq << t.shift) + kAttnQueries - 1) / kAttnQueries);
}
size_t attn_fwd_stat_bytes(const AttnFwdPlan &t) {
  return size_t(t.tail) * t.segments * kAttnQueries * sizeof(float2);
}
size_t attn_fwd_part_bytes(const AttnFwdPlan &t, int D) {
  return size_t(t.tail) * t.segments * kAttnQueries * (D <= 64 ? 64 : 128) * sizeof(float);
}

cudaError_t launch_attn_fwd(const AttnArgs &a, const AttnMaps &m, const AttnFwdPlan &t, void *stat,
                            void *part, int sms, cudaStream_t s) {
  const Params p{a, m, items_of(a, t), t,
                 static_cast<float2 *>(stat), static_cast<float4 *>(part)};
  const bool cap = a.cap > 0.f, bias = a.slopes != nullptr;
  if (a.D <= 64)
    return cap ? (bias ? launch<64, true, true>(p, sms, s) : launch<64, true, false>(p, sms, s))
               : (bias ? launch<64, false, true>(p, sms, s) : launch<64, false, false>(p, sms, s));
  return cap ? (bias ? launch<128, true, true>(p, sms, s) : launch<128, true, false>(p, sms, s))
             : (bias ? launch<128, false, true>(p, sms, s) : launch<128, false, false>(p, sms, s));
}
cudaError_t launch_attn_fwd_join(const AttnArgs &a, const AttnFwdPlan &t, const void *stat,
                                 const void *part, cudaStream_t s) {
  const Params p{a, {}, items_of(a, t), t,
                 static_cast<float2 *>(const_cast<void *>(stat)),
                 static_cast<float4 *>(const_cast<void *>(part))};
  const int cols = a.D <= 64 ? 2 : 4;
  return launch_pdl(a.D <= 64 ? k_attn_fwd_join<64> : k_attn_fwd_join<128>,
                    dim3(static_cast<unsigned>(t.tail) * (kAttnQueries / 32) * cols),
                    dim3(32 * kJoinWarps), 0, s, p);
}

}  // namespace lora
