// norm.cuh -- what the norm's kernels share: a row's elements among its threads,
// sums over them, the weight, and the ring of bulk copies (norm_fwd.cu,
// norm_bwd.cu; norm.cu has the C entry points).
#pragma once

#include <atomic>

#include "dropout.cuh"
#include "host.h"
#include "ptx.cuh"

namespace lora {

constexpr int kMaxDim = 32768;  // 1024 threads x 4 vectors x 8
constexpr int kSmallBlock = 128;  // threads of a block where a group is a warp or less

struct NormRows {  // where row r begins
  int64_t outer, inner;
};

// Rows of an outer entry, and what divides a row's number by them: the quotient of
// a 31-bit number by a constant is a product and a shift (Granlund and Montgomery,
// 1994).
struct NormInner {
  uint32_t n, mul;
  int shift;
};
inline NormInner norm_inner(int64_t n) {
  int l = 0;
  while ((int64_t(1) << l) < n) ++l;
  return {static_cast<uint32_t>(n), static_cast<uint32_t>((uint64_t(1) << (31 + l)) / n + 1), 31 + l};
}

// The addresses between which a tensor's elements lie.
struct NormSpan {
  uint64_t first, last;
};

struct NormFwdArgs {
  const void *x, *res, *w;
  void *h, *y;
  float *rstd, *scale;
  uint8_t *codes;
  NormRows sx, sr, sh, sy;
  NormSpan span_x, span_r;
  int64_t rows;
  NormInner inner;
  int dim, group, w32;
  float eps, inv_dim;
  int dropped;
  DropArgs drop;
};

struct NormBwdArgs {
  const void *dy, *h, *w, *dh;
  const float *rstd;
  void *dx, *dres;
  float *partial;  // [blocks][dim], or null
  NormRows sdy, sh, sdh, sdx, sdr;
  NormSpan span_y, span_h, span_d;
  int64_t rows;
  NormInner inner;
  int dim, group, w32;
  float inv_dim;
  int dropped;
  DropArgs drop;
};

// At the start of a ring's shared memory.
struct RingHead {
  uint64_t full[4];
  int abort_flag;
};
constexpr int kRingHead = 64, kRingRoom = 2048;

// Vectors a thread.  A row's work is one chain through its threads (read, sum,
// barrier, write), so that two vectors a thread and twice the threads take it
// sooner than four, at as many bytes on their way.
constexpr int kRingVectors = 2;

// How a call runs.
struct NormSplit {
  bool ring, heads, shifted;
  int group, vpt, nr, block, per_block;  // threads and vectors of a row; rows at a time
  int stages, blocks_sm;                 // of the ring
  uint32_t buffer;                       // bytes of a row in the ring
};
constexpr int kSms = 152;
constexpr int kRingSmem = 220 * 1024;  // of an SM's, left to its blocks' rings
// How a row lies among its threads: kLoose, its elements one by one; kAligned, vectors;
// kShifted, vectors of rows off the 16-byte boundaries (the ring's only).
constexpr int kLoose = 0, kAligned = 1, kShifted = 2;

// The ring's blocks on an SM, by their threads: at 80 registers a thread, or 128 (96
// in blocks of over 256 threads) where rows are not aligned (at 80 they spill: 5331 x
// 2001 in fp32, both directions, took 114 us instead of 80).
// Shifted rows of fp32: one over 256 threads (two spill: 4096 x 4095 backward, 77 us).
__host__ __device__ constexpr int ring_blocks(int threads, int lay, int es) {
  const bool vec = lay == kAligned || (lay == kShifted && es == 2);
  if (lay == kShifted && !vec && threads > 256) return 1;
  return threads <= 256 ? (vec ? 768 : 512) / threads : threads <= (vec ? 384 : 320) ? 2 : 1;
}

// Narrow rows that a group has on their way at once straight into registers (four
// whose elements come one by one take all of them).
__host__ __device__ constexpr int narrow_rows(bool vec) { return vec ? 4 : 2; }

// Vectors a thread of a narrow aligned row: the sums over its threads, which cost as
// much as the vectors, are over few (131072 rows of 128, forward: one vector a thread
// and four rows 21.7 us, two and two 15.5, four 13.9; of 96, 20.5, 16.2, and three
// 14.7).  Three or `most`, whichever leaves fewer places idle.
inline int narrow_vectors(int vectors, int most) {
  auto places = [&](int n) {
    int lanes = 1;
    while (lanes * n < vectors) lanes *= 2;
    return lanes * n;
  };
  return places(3) < places(most) ? 3 : most;
}
// The ring's threads of narrow rows on an SM, whose registers hold two vectors each, or
// three (four spill, and two at 768 threads).
__host__ __device__ constexpr int heads_threads(int vpt) { return vpt == 2 ? 640 : 512; }

// Few rows (two an SM at most): as many threads as there are vectors.
inline bool norm_few_rows(int64_t rows) { return rows <= 2 * kSms; }

// tensors: that are read a row.
inline NormSplit norm_split(int dim, int64_t rows, int es, int tensors, bool vec, bool backward,
                            bool codes = false, bool shifted = false) {
  const bool wide_codes = codes && es == 4;  // (codes of fp32 rows: not over the ring)
  NormSplit s = {};
  const int vectors = (dim + (shifted ? 14 : 7)) / 8;
  s.nr = 1;
  if (norm_few_rows(rows) && vectors <= 1024) {
    s.vpt = 1;
  } else if (dim > (vec && !backward ? 1024 : 512)) {
    s.vpt = kRingVectors;
    s.group = s.block = ((vectors + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.per_block = 1;
    // (a row may begin and end inside 16 bytes)
    s.buffer = static_cast<uint32_t>((dim * es + 15) / 16 * 16 + (shifted && es == 4 ? 32 : 16));
    const int stage = static_cast<int>(s.buffer) * tensors;
    s.shifted = shifted;
    s.blocks_sm = ring_blocks(s.block, vec ? kAligned : shifted ? kShifted : kLoose, es);
    if (s.blocks_sm > 12) s.blocks_sm = 12;
    for (; s.blocks_sm > 0; --s.blocks_sm) {
      s.stages = (kRingSmem / s.blocks_sm - 1024 - kRingHead - (shifted ? kRingRoom : 0)) / stage;
      if (s.stages >= 2) break;
    }
    s.ring = s.blocks_sm > 0 && s.block <= 512 && !wide_codes;
    if (s.stages > 4) s.stages = 4;
    if (s.ring) return s;
    s.vpt = 4;
  } else {
    s.vpt = vec && vectors >= 6 ? narrow_vectors(vectors, 4) : vectors > 32 ? 4 : 1;
    if (s.vpt == 1) s.nr = narrow_rows(vec);
  }
  const int threads = (vectors + s.vpt - 1) / s.vpt;
  if (threads <= 32) {
    s.group = 1;
    while (s.group < threads) s.group *= 2;
    s.block = kSmallBlock;
  } else {
    s.group = s.block = (threads + 31) / 32 * 32;
  }
  s.per_block = s.block / s.group * s.nr;
  return s;
}

// The backward's narrow rows of which `inner` lie side by side in every tensor, as the
// ring's rows: each of whole vectors, on 1, 2, 4 ... 32 threads.  False: not so.
inline bool norm_heads(int dim, int64_t outer, int64_t inner, int es, int tensors, NormSplit &s) {
  const int vectors = dim / 8;
  const int64_t wide = inner * dim;
  if (dim % 8 != 0 || vectors < 6 || inner < 2 || wide <= 1024 || wide > 8192 || norm_few_rows(outer)) return false;
  NormSplit t = {};
  t.heads = true;
  t.vpt = narrow_vectors(vectors, 2);
  t.group = 1;
  while (t.group * t.vpt < vectors) t.group *= 2;
  t.block = static_cast<int>((inner * t.group + 31) / 32 * 32);
  if (t.group > 32 || t.block > 256) return false;
  t.nr = t.per_block = 1;
  t.buffer = static_cast<uint32_t>(wide * es);
  t.blocks_sm = heads_threads(t.vpt) / t.block;
  if (t.blocks_sm > 12) t.blocks_sm = 12;
  for (; t.blocks_sm > 0; --t.blocks_sm) {
    t.stages = (kRingSmem / t.blocks_sm - 1024 - kRingHead) / (static_cast<int>(t.buffer) * tensors);
    if (t.stages >= 2) break;
  }
  if (t.blocks_sm == 0) return false;
  if (t.stages > 4) t.stages = 4;
  s = t;
  return true;
}

// Blocks of the backward, each with a line of partial sums.
inline int norm_bwd_blocks(const NormSplit &s, int64_t rows) {
  const int64_t n = (rows + s.per_block - 1) / s.per_block;
  const int most = kSms * (s.ring || s.heads ? s.blocks_sm : 4);
  return static_cast<int>(n < most ? n : most);
}

// Whether a ring's rows can be taken as kShifted: each tensor as far past a 16-byte
// boundary as the others, row by row, and bf16 weights with bf16 rows.
struct NormShift {
  uint64_t at = 0;
  int64_t step = 0;
  bool any = false, ok = true;
  // (rows of an input nearer than 16 bytes would end past the tensor with their last 16)
  void add(const void *p, int64_t stride, int es) {
    const uint64_t here = reinterpret_cast<uint64_t>(p) % 16;
    if (any && (here != at || (stride - step) % (16 / es) != 0)) ok = false;
    if ((stride < 0 ? -stride : stride) < 16 / es) ok = false;
    if (!any) at = here, step = stride, any = true;
  }
};

cudaError_t launch_norm_fwd(lora_dtype_t dtype, bool vec, const NormFwdArgs &a, const NormSplit &s, int tensors,
                            unsigned *status, cudaStream_t st);
cudaError_t launch_norm_bwd(lora_dtype_t dtype, bool vec, const NormBwdArgs &a, const NormSplit &s, int tensors,
                            unsigned *status, cudaStream_t st);
// dw from the blocks' lines of sums (fp32: of that type, else bf16).
cudaError_t launch_norm_dw(bool fp32, const float *partial, int blocks, int dim, void *dw, cudaStream_t st);

namespace {

struct Where {
  int64_t o, i;
  __device__ __forceinline__ int64_t at(const NormRows &s) const { return o * s.outer + i * s.inner; }
};
__device__ __forceinline__ Where where(int64_t row, const NormInner &inner) {
  const uint32_t r = static_cast<uint32_t>(row);  // below 2^31
  if (inner.n == 1) return {row, 0};
  const uint32_t o = static_cast<uint32_t>(uint64_t(r) * inner.mul >> inner.shift);
  return {static_cast<int64_t>(o), static_cast<int64_t>(r - o * inner.n)};
}

// A row belongs to `group` threads, VPT vectors of eight elements each.  kAligned:
// eight that lie side by side (vector t + j group).  kLoose: eight that lie `group`
// apart, so that a warp's accesses cover neighbours.  kShifted: as kAligned, counted
// from the 16-byte boundary that is m elements before the row (the first and the last
// vector hold some elements of it).
template <int AL>
__device__ __forceinline__ int element(int t, int group, int j, int k) {
  return AL != kLoose ? (t + j * group) * 8 + k : (j * 8 + k) * group + t;
}
// Thread t's vectors of a row of `dim` elements at p; zeros past its end.
template <int AL, class T, int VPT>
__device__ __forceinline__ void fetch(Raw8<T> (&v)[VPT], const T *p, int t, int group, int dim) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if constexpr (AL) {
      const int c = (t + j * group) * 8;
      if (c < dim) {
        v[j].load(p + c);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j].set(i, both(0.f));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = element<false>(t, group, j, k);
        if (k % 2 == 0) v[j].set(k / 2, both(0.f));
        if (c < dim) v[j].load1(k, p + c);
      }
    }
  }
}
// Which elements of a thread's vector are the shifted row's: a bit each.
template <int VPT>
__device__ __forceinline__ void own_bits(uint32_t (&own)[VPT], int t, int group, int dim, int m) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = (t + j * group) * 8 - m;
    own[j] = c >= dim ? 0u : (c < 0 ? 255u << -c : 255u) & (c + 8 > dim ? 255u >> (c + 8 - dim) : 255u) & 255u;
  }
}
__device__ __forceinline__ void keep_only(Raw8<__nv_bfloat16> &v, uint32_t own) {
  own |= own << 15;  // elements 2 i and 2 i + 1 at bits 2 i and 16 + 2 i
#pragma unroll
  for (int i = 0; i < 4; ++i) v.u[i] &= (own >> 2 * i & 0x10001u) * 0xffffu;
}
__device__ __forceinline__ void keep_only(Raw8<float> &v, uint32_t own) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.f[i] = make_float2(own >> 2 * i & 1u ? v.f[i].x : 0.f, own >> 2 * i & 2u ? v.f[i].y : 0.f);
}
// The same of a row off the boundaries, one by one; zeros before and past it.
template <class T, int VPT>
__device__ __forceinline__ void fetch_cut(Raw8<T> (&v)[VPT], const T *p, int t, int group, int dim, int m) {
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<kShifted>(t, group, j, k) - m;
      if (k % 2 == 0) v[j].set(k / 2, both(0.f));
      if (c >= 0 && c < dim) v[j].load1(k, p + c);
    }
}
// (m, own: of shifted rows)
template <int AL, class T>
__device__ __forceinline__ void put(T *p, const Raw8<T> &v, int t, int group, int j, int dim, int m = 0,
                                    uint32_t own = 255u) {
  if constexpr (AL == kShifted) {
    T *to = p + ((t + j * group) * 8 - m);
    if (own == 255u) {
      v.store(to);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (own >> k & 1u) v.store1(k, to + k);
    }
  } else if constexpr (AL == kAligned) {
    const int c = (t + j * group) * 8;
    if (c < dim) v.store(p + c);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<false>(t, group, j, k);
      if (c < dim) v.store1(k, p + c);
    }
  }
}
template <int AL, class T>
__device__ __forceinline__ void put(T *p, const float2 (&v)[4], int t, int group, int j, int dim, int m = 0,
                                    uint32_t own = 255u) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.set(i, v[i]);
  put<AL>(p, r, t, group, j, dim, m, own);
}
// Drops out vector j.  Where a thread's elements lie `group` apart (a multiple of
// 32), a warp's 32 neighbours take the words of eight calls of the generator: each
// lane makes one of those of four steps, and hands the words round.
template <int AL>
__device__ __forceinline__ void drop_vector(const DropArgs &d, const DropNow &now, int64_t row, int t,
                                            int group, int j, float2 (&v)[4]) {
  if constexpr (AL) {
    drop8(d, now, static_cast<uint32_t>(t + j * group), row, v);
  } else if (group >= 32) {
    const int lane = t & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = element<false>(t - lane, group, j, 4 * h + (lane >> 3)) + 4 * (lane & 7);
      const uint4 w = drop_words(d, now, static_cast<uint32_t>(c) >> 2, row);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int from = 8 * k + (lane >> 2);
        const uint4 all = make_uint4(__shfl_sync(0xffffffffu, w.x, from), __shfl_sync(0xffffffffu, w.y, from),
                                     __shfl_sync(0xffffffffu, w.z, from), __shfl_sync(0xffffffffu, w.w, from));
        float &x = k & 1 ? v[2 * h + k / 2].y : v[2 * h + k / 2].x;
        x = drop1(d, word_of(all, lane & 3), x);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = static_cast<uint32_t>(element<false>(t, group, j, k));
      const uint4 w = drop_words_of(now.seed, c >> 2, static_cast<uint32_t>(row),
                                    static_cast<uint32_t>(uint64_t(row) >> 32), now.offset);
      float &x = k & 1 ? v[k / 2].y : v[k / 2].x;
      x = drop1(d, word_of(w, c & 3), x);
    }
  }
}

// The weight: kept in registers where it is bf16 and KEEP, else read again for each
// row (from L1: it is the only thing that is read through it).  Always kept where rows
// are shifted.
template <int AL, bool KEEP, class T, int VPT>
struct Weight {
  static constexpr bool kKeep = KEEP && (sizeof(T) == 2 || AL == kShifted);
  Raw8<T> kept[kKeep ? VPT : 1];
  const void *from;
  bool wide;  // fp32
  __device__ __forceinline__ Weight(const void *w, int w32, int t, int group, int dim, int m = 0)
      : from(w), wide(AL != kShifted && (sizeof(T) == 4 || w32 != 0)) {
    if constexpr (kKeep && AL == kShifted) {
      fetch_cut(kept, static_cast<const T *>(w), t, group, dim, m);
    } else if constexpr (kKeep) {
      if (!wide) fetch<AL>(kept, static_cast<const T *>(w), t, group, dim);
    }
  }
  template <class S>
  __device__ __forceinline__ void read(const S *w, int j, int t, int group, int dim, float2 (&u)[4]) const {
    Raw8<S> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.set(i, both(0.f));
    if constexpr (AL == kAligned) {
      const int c = (t + j * group) * 8;
      if (c < dim) o.load(w + c);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = element<false>(t, group, j, k);
        if (c < dim) o.load1(k, w + c);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = o.pair(i);
  }
  __device__ __forceinline__ void get(int j, int t, int group, int dim, float2 (&u)[4]) const {
    if (wide) {
      read(static_cast<const float *>(from), j, t, group, dim, u);
    } else if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = VPT == 1 ? kept[j].pair(i) : kept[j].again(i);
    } else {
      read(static_cast<const T *>(from), j, t, group, dim, u);
    }
  }
};

// Sum (or largest) over the `group` threads of a row, the same bits in each of
// them: shuffles, and for a group of several warps (then it is the block) one
// barrier.  slot: 32 floats that are 0 beyond the block's warps, others than
// those of the last call.
template <bool MAX>
__device__ __forceinline__ float over_group(float v, int group, float *slot) {
  const int lanes = group < 32 ? group : 32;
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if (group <= 32) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const float4 *all = reinterpret_cast<const float4 *>(slot);
  v = 0.f;
  for (int i = 0; i < group; i += 128) {
    const float4 q = all[i >> 7];
    v = MAX ? fmaxf(fmaxf(v, fmaxf(q.x, q.y)), fmaxf(q.z, q.w)) : v + ((q.x + q.y) + (q.z + q.w));
  }
  return v;
}
__device__ __forceinline__ void clear_slots(float *slots, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) slots[i] = 0.f;
}

// How far a shifted row begins past a boundary; the same for all rows of a block whose
// step is a multiple of eight.
template <class T>
__device__ __forceinline__ int row_shift(const T *row) {
  return static_cast<int>(reinterpret_cast<uint64_t>(row) / sizeof(T) % (16 / sizeof(T)));
}
// ---- the ring ----
// Stage s of it holds one row of each tensor, a buffer apart; bulk copies fill it
// and count on full[s].  A copy takes whole 16-byte units: of a row that does not
// begin or end on one, also the neighbours' bytes, which lie between the
// tensor's first and last element for all but the first and the last row; what
// these two miss comes straight from memory.

template <class T>
struct RowCopy {
  const T *src;
  int lead, lo, hi;  // elements before the row in the buffer; the row's copied ones
  __device__ __forceinline__ uint32_t bytes() const {
    return static_cast<uint32_t>(hi + (lo > 0 ? -lo : lead)) * static_cast<uint32_t>(sizeof(T));
  }
};
// first, last: the addresses between which the tensor lies.
template <int AL, class T>
__device__ __forceinline__ RowCopy<T> row_copy(const T *src, int dim, const NormSpan &span) {
  RowCopy<T> c = {src, 0, 0, dim};
  if constexpr (AL != kAligned) {
    const uint64_t a = reinterpret_cast<uint64_t>(src), end = a + uint64_t(dim) * sizeof(T);
    uint64_t lo = a & ~uint64_t(15), hi = (end + 15) & ~uint64_t(15);
    c.lead = static_cast<int>((a - lo) / sizeof(T));
    if (lo < span.first) {
      lo += 16;
      c.lo = static_cast<int>((lo - a) / sizeof(T));
    }
    if (hi > span.last) hi -= 16;
    c.hi = hi > lo ? static_cast<int>((int64_t(hi) - int64_t(a)) / int64_t(sizeof(T))) : c.lo - c.lead;
    if (hi <= lo) {  // nothing between two boundaries
      c.lo = c.hi = 0;
      c.lead = 0;
    }
  }
  return c;
}
template <class T>
__device__ __forceinline__ void copy_start(const RowCopy<T> &c, uint32_t buf, uint32_t bar) {
  const uint32_t n = c.bytes();
  // (where the first unit is left out, its place in the buffer stays empty)
  if (n > 0) bulk_load(buf + (c.lo > 0 ? 16u : 0u), c.src + (c.lo > 0 ? c.lo : -c.lead), n, bar);
}
// Thread t's vectors of a row that has arrived in buf.
template <int AL, class T, int VPT>
__device__ __forceinline__ void take(Raw8<T> (&v)[VPT], const RowCopy<T> &c, const uint8_t *buf, int t,
                                     int group, int dim) {
  const T *in = reinterpret_cast<const T *>(buf) + c.lead;
  if constexpr (AL == kAligned) {
    fetch<true>(v, in, t, group, dim);
  } else if (c.lo <= 0 && c.hi >= dim) {
    fetch<false>(v, in, t, group, dim);
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = element<false>(t, group, j, k);
        if (k % 2 == 0) v[j].set(k / 2, both(0.f));
        if (e < dim) v[j].load1(k, e >= c.lo && e < c.hi ? in + e : c.src + e);
      }
  }
}

// Waits for stage s of row i of this block's; the abort flag is up once a wait
// ran out.
__device__ __forceinline__ void ring_wait(RingHead *head, int s, uint32_t phase, unsigned *status) {
  mbar_wait(smem_u32(&head->full[s]), phase, &head->abort_flag, status);
}
// On the way out: the copies in flight land first.
__device__ __forceinline__ void ring_drain(RingHead *head, int s, uint32_t phase, int rows, int stages) {
  for (; rows > 0; --rows) {
    mbar_wait_drain(smem_u32(&head->full[s]), phase);
    if (++s == stages) s = 0, phase ^= 1u;
  }
}
// Shifted rows: all copies of a block are of `bytes` from the boundary before a row,
// but those of the tensor's first and last row, which may not reach so far (row_copy).
struct ShiftCopy {
  int m;
  uint32_t bytes;
  int64_t rows;
  template <class T>
  __device__ __forceinline__ static ShiftCopy of(const T *row, int dim, int64_t rows) {
    const int m = row_shift(row);
    return {m, static_cast<uint32_t>((m + dim) * int(sizeof(T)) + 15) / 16 * 16, rows};
  }
  __device__ __forceinline__ bool whole(int64_t row) const { return row > 0 && row < rows - 1; }
};
template <class T>
__device__ __forceinline__ uint32_t copy_bytes(const ShiftCopy &c, const T *src, int64_t row, int dim,
                                               const NormSpan &span) {
  return c.whole(row) ? c.bytes : row_copy<kShifted>(src, dim, span).bytes();
}
template <class T>
__device__ __forceinline__ void copy_start(const ShiftCopy &c, const T *src, int64_t row, int dim,
                                           const NormSpan &span, uint32_t buf, uint32_t bar) {
  if (c.whole(row))
    bulk_load(buf, src - c.m, c.bytes, bar);
  else
    copy_start(row_copy<kShifted>(src, dim, span), buf, bar);
}
// Thread t's vectors, as they lie around the row too (only_own takes that away).
template <class T, int VPT>
__device__ __forceinline__ void take(Raw8<T> (&v)[VPT], const ShiftCopy &c, const T *src, int64_t row,
                                     const NormSpan &span, const uint8_t *buf, int t, int group, int dim) {
  const T *in = reinterpret_cast<const T *>(buf);
  if (c.whole(row)) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) v[j].load(in + (t + j * group) * 8);  // (there is room behind the ring)
  } else {
    const auto r = row_copy<kShifted>(src, dim, span);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = element<kShifted>(t, group, j, k) - c.m;
        if (k % 2 == 0) v[j].set(k / 2, both(0.f));
        if (e >= 0 && e < dim) v[j].load1(k, e >= r.lo && e < r.hi ? in + (c.m + e) : src + e);
      }
  }
}
template <class T, int VPT>
__device__ __forceinline__ void only_own(Raw8<T> (&v)[VPT], const uint32_t (&own)[VPT]) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) keep_only(v[j], own[j]);
}
template <int VPT>
__device__ __forceinline__ bool all_own(const uint32_t (&own)[VPT]) {
  uint32_t u = 255u;
#pragma unroll
  for (int j = 0; j < VPT; ++j) u &= own[j];
  return u == 255u;
}
__device__ __forceinline__ void ring_init(RingHead *head, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&head->full[s]), 1);
    head->abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// `allowed`: of this kernel.  (Its limit is said once, for every call's size: host threads
// whose calls differ in it would lower it under one another's launches.)
template <class... P, class A>
cudaError_t launch_ring(void (*kern)(P...), std::atomic<uint64_t> &allowed, int blocks, const NormSplit &s,
                        int tensors, const A &a, unsigned *status, cudaStream_t st) {
  // (threads past the end of a shifted row read on, by 2 KB at most; the SM has it left)
  const size_t smem = kRingHead + size_t(s.stages) * tensors * s.buffer + (s.shifted ? kRingRoom : 0);
  const cudaError_t e = allow_smem(kern, kRingSmem, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(blocks), dim3(s.block), smem, st, a, s.stages, s.buffer, status);
}

}  // namespace
}  // namespace lora
