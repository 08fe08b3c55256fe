// norm.cu -- root-mean-square norm with the residual's addition, dropout of the
// branch and an 8-bit output (include/lora_norm.h; ch05 "Acceleration
// principles: Triton kernels and fused LoRA", §5.4: one pass over the row).
//
// A row stays in the registers of the threads that read it: it is read once,
// its sum of squares (and largest magnitude) go through shuffles and shared
// memory, and it is written once.  Bound by memory: what counts is how many bytes
// an SM has on their way.
//
// Two forms.  Rows wider than 1024 elements, and more than the SMs take at once:
// blocks stay, and bulk copies bring the next rows into a ring in shared memory
// while one is worked on (k_norm_fwd_ring, k_norm_bwd_ring).  Narrow rows, several
// a warp, and few rows, where latency counts: straight into registers (k_norm_fwd,
// k_norm_bwd).
#include <climits>
#include <initializer_list>

#include "dropout.cuh"
#include "e4m3.cuh"
#include "host.h"
#include "lora_norm.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kMaxDim = 32768;  // 1024 threads x 4 vectors x 8
constexpr int kSmallBlock = 128;  // threads of a block where a group is a warp or less

struct Rows {  // where row r begins
  int64_t outer, inner;
};

// The addresses between which a tensor's elements lie.
struct Span {
  uint64_t first, last;
};

struct FwdArgs {
  const void *x, *res, *w;
  void *h, *y;
  float *rstd, *scale;
  uint8_t *codes;
  Rows sx, sr, sh, sy;
  Span span_x, span_r;
  int64_t rows;
  uint32_t inner;  // rows an outer entry
  int dim, group, w32;
  float eps;
  int dropped;
  DropArgs drop;
};

struct BwdArgs {
  const void *dy, *h, *w, *dh;
  const float *rstd;
  void *dx, *dres;
  float *partial;  // [blocks][dim], or null
  Rows sdy, sh, sdh, sdx, sdr;
  Span span_y, span_h, span_d;
  int64_t rows;
  uint32_t inner;
  int dim, group, w32;
  int dropped;
  DropArgs drop;
};

struct Where {
  int64_t o, i;
  __device__ __forceinline__ int64_t at(const Rows &s) const { return o * s.outer + i * s.inner; }
};
__device__ __forceinline__ Where where(int64_t row, uint32_t inner) {
  if (inner == 1) return {row, 0};
  const uint32_t r = static_cast<uint32_t>(row);  // below 2^31
  return {static_cast<int64_t>(r / inner), static_cast<int64_t>(r % inner)};
}

// A row belongs to `group` threads, VPT vectors of eight elements each.  Aligned
// rows (AL): eight that lie side by side (vector t + j group).  Others: eight that
// lie `group` apart, so that a warp's accesses cover neighbours.
template <bool AL>
__device__ __forceinline__ int element(int t, int group, int j, int k) {
  return AL ? (t + j * group) * 8 + k : (j * 8 + k) * group + t;
}
// Thread t's vectors of a row of `dim` elements at p; zeros past its end.
template <bool AL, class T, int VPT>
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
template <bool AL, class T>
__device__ __forceinline__ void put(T *p, const Raw8<T> &v, int t, int group, int j, int dim) {
  if constexpr (AL) {
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
template <bool AL, class T>
__device__ __forceinline__ void put(T *p, const float2 (&v)[4], int t, int group, int j, int dim) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.set(i, v[i]);
  put<AL>(p, r, t, group, j, dim);
}
template <bool AL>
__device__ __forceinline__ void drop_vector(const DropArgs &d, const DropNow &now, int64_t row, int t,
                                            int group, int j, float2 (&v)[4]) {
  if constexpr (AL) {
    drop8(d, now, static_cast<uint32_t>(t + j * group), row, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = static_cast<uint32_t>(element<false>(t, group, j, k));
      float &x = k & 1 ? v[k / 2].y : v[k / 2].x;
      x = drop1(d, word_of(drop_words(d, now, c >> 2, row), c & 3), x);
    }
  }
}

// The weight: in bf16 kept in registers, in fp32 (which would take 32 of them)
// read again for each row.
template <bool AL, class T, int VPT>
struct Weight {
  static constexpr bool kKeep = sizeof(T) == 2;
  Raw8<T> kept[kKeep ? VPT : 1];
  const float *wide;
  __device__ __forceinline__ Weight(const void *w, int w32, int t, int group, int dim)
      : wide(kKeep && !w32 ? nullptr : static_cast<const float *>(w)) {
    if constexpr (kKeep)
      if (wide == nullptr) fetch<AL>(kept, static_cast<const T *>(w), t, group, dim);
  }
  __device__ __forceinline__ void get(int j, int t, int group, int dim, float2 (&u)[4]) const {
    if (kKeep && wide == nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = kept[kKeep ? j : 0].again(i);
      return;
    }
    Raw8<float> o[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[0].set(i, both(0.f));
    if constexpr (AL) {
      const int c = (t + j * group) * 8;
      if (c < dim) o[0].load(wide + c);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = element<false>(t, group, j, k);
        if (c < dim) o[0].load1(k, wide + c);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = o[0].pair(i);
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

// r = (ss / dim + eps)^(-1/2) of the row in v.  Where the squares leave the
// range of fp32 the sum is taken again of values scaled down by 2^-70 (exact),
// which the result is scaled by as well.
template <class T, int VPT>
__device__ __forceinline__ float rstd_of(const Raw8<T> (&v)[VPT], int dim, float eps, int group,
                                         float *slot, float *slot2) {
  float2 s = both(0.f);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(v[j].pair(i), v[j].pair(i), s);
  const float ss = over_group<false>(s.x + s.y, group, slot);
  const float n = static_cast<float>(dim);
  // the same in every thread of a block-wide group; the smaller groups of a
  // warp shuffle together
  const bool far = !(ss <= 1e38f);
  if (!(group > 32 ? far : __any_sync(0xffffffffu, far))) return rsqrtf(ss / n + eps);
  float s2 = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = mul2(v[j].pair(i), both(0x1p-70f));
      s2 = fmaf(u.x, u.x, fmaf(u.y, u.y, s2));
    }
  s2 = over_group<false>(s2, group, slot2);
  return far ? 0x1p-70f * rsqrtf(s2 / n + eps * 0x1p-140f) : rsqrtf(ss / n + eps);
}

// x becomes drop(x) + residual, as the stream holds it (rounded once to the
// dtype: the norm is of that), written to h.
template <bool AL, bool DROP, class T, int VPT>
__device__ __forceinline__ void to_stream(const FwdArgs &a, const DropNow &now, Raw8<T> (&x)[VPT],
                                          const Raw8<T> (&res)[VPT], int64_t row, T *h, int t,
                                          int group, int dim) {
  if (!DROP && a.res == nullptr) return;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[j].pair(i);
    if constexpr (DROP) drop_vector<AL>(a.drop, now, row, t, group, j, v);
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], res[j].pair(i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j].set(i, v[i]);
    if (a.h != nullptr) put<AL>(h, x[j], t, group, j, dim);
    if (AL && (t + j * group) * 8 >= dim) {  // (a mask of zeros may have set a sign)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j].set(i, both(0.f));
    }
  }
}

// y = h r w to memory, and the codes and the scale.
template <bool AL, bool FP8, class T, int VPT>
__device__ __forceinline__ void to_outputs(const FwdArgs &a, const Raw8<T> (&h)[VPT],
                                           const Weight<AL, T, VPT> &w, float rstd, int64_t row, T *y,
                                           int t, int group, int dim, float *slot) {
  float2 v[FP8 ? VPT : 1][4];
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 u[4], (&o)[4] = v[FP8 ? j : 0];
    w.get(j, t, group, a.dim, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = mul2(mul2(h[j].pair(i), both(rstd)), u[i]);
      if constexpr (FP8) top = fmaxf(top, fmaxf(fabsf(o[i].x), fabsf(o[i].y)));
    }
    if (a.y != nullptr) put<AL>(y, o, t, group, j, dim);
  }
  if constexpr (FP8) {
    top = over_group<true>(top, group, slot);
    // an infinite row's scale is that of the largest finite number
    const int e = top <= 3.4028234e38f ? max(pow2_exponent(top), -126) : 120;
    const float inv = ldexpf(1.f, -e);
    if (dim > 0 && t == 0) a.scale[row] = ldexpf(1.f, e);
    uint8_t *q = a.codes + row * a.dim;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if constexpr (AL) {
        const int c = (t + j * group) * 8;
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = to_e4m3x2(mul2(v[j][i], both(inv)));
        if (c < dim) *reinterpret_cast<uint2 *>(q + c) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = element<false>(t, group, j, k);
          if (c < dim) q[c] = to_e4m3((k & 1 ? v[j][k / 2].y : v[j][k / 2].x) * inv);
        }
      }
    }
  }
}

// Forward, straight into registers: NR rows a group of threads, all of them on
// their way at once.
template <class T, int VPT, bool AL, bool DROP, bool FP8, int NR, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_fwd(const __grid_constant__ FwdArgs a) {
  __shared__ __align__(16) float slots[96];
  clear_slots(slots, 96);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int group = a.group;
  const int t = threadIdx.x % group, subs = blockDim.x / group;
  const int64_t first = int64_t(blockIdx.x) * (subs * NR) + threadIdx.x / group;
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  Raw8<T> hx[NR][VPT], hr[NR][VPT];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int64_t row = first + n * subs;
    const int dim = row < a.rows ? a.dim : 0;  // a group without a row holds zeros
    const Where at = where(row < a.rows ? row : 0, a.inner);
    fetch<AL>(hx[n], static_cast<const T *>(a.x) + at.at(a.sx), t, group, dim);
    if (a.res != nullptr) fetch<AL>(hr[n], static_cast<const T *>(a.res) + at.at(a.sr), t, group, dim);
  }
  const Weight<AL, T, VPT> w(a.w, a.w32, t, group, a.dim);
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int64_t row = first + n * subs;
    const bool live = row < a.rows;
    const int dim = live ? a.dim : 0;
    const Where at = where(live ? row : 0, a.inner);
    to_stream<AL, DROP>(a, now, hx[n], hr[n], row, static_cast<T *>(a.h) + at.at(a.sh), t, group, dim);
    const float rstd = rstd_of(hx[n], a.dim, a.eps, group, slots, slots + 32);
    if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    to_outputs<AL, FP8>(a, hx[n], w, rstd, row, static_cast<T *>(a.y) + at.at(a.sy), t, group, dim,
                        slots + 64);
  }
}

// ---- the ring ----
// Vectors a thread: as many as its registers hold (the forward's 80, the
// backward's 128); the fewer threads a row, the fewer instructions it takes to
// add up their sums.
__host__ __device__ constexpr int ring_vectors(int es) { return es == 2 ? 4 : 2; }

// Stage s of it holds one row of each tensor, a buffer apart; bulk copies fill it
// and count on full[s].  A copy takes whole 16-byte units: of a row that does not
// begin or end on one, also the neighbours' bytes, which lie between the
// tensor's first and last element for all but the first and the last row; what
// these two miss comes straight from memory.
struct RingHead {
  uint64_t full[4];
  int abort_flag;
};
constexpr int kRingHead = 64;

template <class T>
struct RowCopy {
  const T *src;
  int lead, lo, hi;  // elements before the row in the buffer; the row's copied ones
  __device__ __forceinline__ uint32_t bytes() const {
    return static_cast<uint32_t>(hi + (lo > 0 ? -lo : lead)) * static_cast<uint32_t>(sizeof(T));
  }
};
// first, last: the addresses between which the tensor lies.
template <bool AL, class T>
__device__ __forceinline__ RowCopy<T> row_copy(const T *src, int dim, const Span &span) {
  RowCopy<T> c = {src, 0, 0, dim};
  if constexpr (!AL) {
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
template <bool AL, class T, int VPT>
__device__ __forceinline__ void take(Raw8<T> (&v)[VPT], const RowCopy<T> &c, const uint8_t *buf, int t,
                                     int group, int dim) {
  const T *in = reinterpret_cast<const T *>(buf) + c.lead;
  if constexpr (AL) {
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
__device__ __forceinline__ void ring_init(RingHead *head, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&head->full[s]), 1);
    head->abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// Forward over the ring: block b takes rows b, b + grid, ...
template <class T, bool AL, bool DROP, bool FP8, int MAX, int BLOCKS>
__global__ void __launch_bounds__(MAX, BLOCKS)
    k_norm_fwd_ring(const __grid_constant__ FwdArgs a, int stages, uint32_t buffer, unsigned *status) {
  constexpr int VPT = ring_vectors(sizeof(T));
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float slots[128];
  auto *head = reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + kRingHead;
  clear_slots(slots, 128);
  ring_init(head, stages);
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  const int group = blockDim.x, t = threadIdx.x, tensors = a.res != nullptr ? 2 : 1;
  auto copy_x = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.x) + at.at(a.sx), a.dim, a.span_x);
  };
  auto copy_r = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.res) + at.at(a.sr), a.dim, a.span_r);
  };
  auto start = [&](int64_t row, int s) {
    const Where at = where(row, a.inner);
    const uint32_t bar = smem_u32(&head->full[s]), buf = smem_u32(ring + s * tensors * buffer);
    const auto cx = copy_x(at);
    if (tensors == 2) {
      const auto cr = copy_r(at);
      mbar_expect_tx(bar, cx.bytes() + cr.bytes());
      copy_start(cr, buf + buffer, bar);
    } else {
      mbar_expect_tx(bar, cx.bytes());
    }
    copy_start(cx, buf, bar);
  };
  const int64_t step = gridDim.x;
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < a.rows) start(blockIdx.x + i * step, i);
  const Weight<AL, T, VPT> w(a.w, a.w32, t, group, a.dim);
  int s = 0, parity = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += step) {
    const int t = each_time(int(threadIdx.x));
    const Where at = where(row, a.inner);
    Raw8<T> x[VPT];
    ring_wait(head, s, phase, status);
    {
      const uint8_t *buf = ring + s * tensors * buffer;
      Raw8<T> r[VPT];
      take<AL>(x, copy_x(at), buf, t, group, a.dim);
      if (tensors == 2) take<AL>(r, copy_r(at), buf + buffer, t, group, a.dim);
      to_stream<AL, DROP>(a, now, x, r, row, static_cast<T *>(a.h) + at.at(a.sh), t, group, a.dim);
    }
    // its barrier: every thread has read the stage
    const float rstd = rstd_of(x, a.dim, a.eps, group, slots + 32 * parity, slots + 64);
    parity ^= 1;
    if (*static_cast<volatile int *>(&head->abort_flag)) {  // a copy that never came
      const int64_t left = (a.rows - row + step - 1) / step;
      if (t == 0) ring_drain(head, s, phase, static_cast<int>(left < stages ? left : stages), stages);
      return;
    }
    if (t == 0) {
      if (row + stages * step < a.rows) start(row + stages * step, s);
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if (++s == stages) s = 0, phase ^= 1u;
    to_outputs<AL, FP8>(a, x, w, rstd, row, static_cast<T *>(a.y) + at.at(a.sy), t, group, a.dim,
                        slots + 96);
  }
}

// ---- backward ----
// What a row's threads do with it: g = dy w and h r, their mean product, then
// d = r (g - h r mean) + dh, dropped out where the branch was.
template <bool AL, bool DROP, class T, int VPT>
__device__ __forceinline__ void row_backward(const BwdArgs &a, const DropNow &now,
                                             const Raw8<T> (&hy)[VPT], const Raw8<T> (&hh)[VPT],
                                             const Raw8<T> (&hd)[VPT], const Weight<AL, T, VPT> &w,
                                             float rstd, int64_t row, const Where &at, int t, int group,
                                             int dim, float *slot, float2 (&acc)[VPT][4]) {
  float2 s = both(0.f);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 u[4];
    w.get(j, t, group, a.dim, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 hat = mul2(hh[j].pair(i), both(rstd)), y = hy[j].pair(i);
      acc[j][i] = fma2(y, hat, acc[j][i]);
      s = fma2(mul2(y, u[i]), hat, s);
    }
  }
  const float along = over_group<false>(s.x + s.y, group, slot) / static_cast<float>(a.dim);
  const float2 back = both(-along * rstd * rstd);  // d = r g - h (r^2 mean) + dh
  T *dx = static_cast<T *>(a.dx) + at.at(a.sdx);
  T *dres = static_cast<T *>(a.dres) + at.at(a.sdr);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 d[4], u[4];
    w.get(j, t, group, a.dim, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = mul2(hh[j].pair(i), back);
      d[i] = fma2(mul2(hy[j].pair(i), u[i]), both(rstd), d[i]);
      if (a.dh != nullptr) d[i] = add2(d[i], hd[j].pair(i));
    }
    if (a.dres != nullptr) put<AL>(dres, d, t, group, j, dim);
    if constexpr (DROP) drop_vector<AL>(a.drop, now, row, t, group, j, d);
    put<AL>(dx, d, t, group, j, dim);
  }
}

// Straight into registers: blocks stay and take NR rows a group at a time; each
// thread adds up dy h r of its columns over the rows that it took.
template <class T, int VPT, bool AL, bool DROP, int NR, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_bwd(const __grid_constant__ BwdArgs a) {
  __shared__ __align__(16) float slots[64];
  __shared__ float cols[kSmallBlock * VPT * 8];  // dw of the groups of a small block
  clear_slots(slots, 64);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  const int group = a.group;
  const int t = threadIdx.x % group, sub = threadIdx.x / group, subs = blockDim.x / group;
  float2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  const Weight<AL, T, VPT> w(a.w, a.w32, t, group, a.dim);
  int parity = 0;
  const int64_t step = int64_t(gridDim.x) * subs * NR;
  for (int64_t first = int64_t(blockIdx.x) * subs * NR; first < a.rows; first += step) {
    const int t = each_time(int(threadIdx.x % group));
    Raw8<T> hy[NR][VPT], hh[NR][VPT], hd[NR][VPT];
    float rstd[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int64_t row = first + n * subs + sub;
      const bool live = row < a.rows;
      const int dim = live ? a.dim : 0;
      const Where at = where(live ? row : 0, a.inner);
      fetch<AL>(hy[n], static_cast<const T *>(a.dy) + at.at(a.sdy), t, group, dim);
      fetch<AL>(hh[n], static_cast<const T *>(a.h) + at.at(a.sh), t, group, dim);
      if (a.dh != nullptr) fetch<AL>(hd[n], static_cast<const T *>(a.dh) + at.at(a.sdh), t, group, dim);
      rstd[n] = live ? a.rstd[row] : 0.f;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int64_t row = first + n * subs + sub;
      const bool live = row < a.rows;
      row_backward<AL, DROP>(a, now, hy[n], hh[n], hd[n], w, rstd[n], row,
                             where(live ? row : 0, a.inner), t, group, live ? a.dim : 0,
                             slots + 32 * parity, acc);
      parity ^= 1;
    }
  }
  if (a.partial == nullptr) return;
  float *out = a.partial + int64_t(blockIdx.x) * a.dim;
  const int width = group * VPT * 8;  // >= dim
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<AL>(t, group, j, k);
      const float v = k & 1 ? acc[j][k / 2].y : acc[j][k / 2].x;
      if (subs > 1)
        cols[sub * width + c] = v;
      else if (c < a.dim)
        out[c] = v;
    }
  }
  if (subs == 1) return;
  __syncthreads();  // several rows at a time: the groups' sums, added in their order
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
    float s = 0.f;
    for (int i = 0; i < subs; ++i) s += cols[i * width + c];
    out[c] = s;
  }
}

// Over the ring.
template <class T, bool AL, bool DROP, int MAX, int BLOCKS>
__global__ void __launch_bounds__(MAX, BLOCKS)
    k_norm_bwd_ring(const __grid_constant__ BwdArgs a, int stages, uint32_t buffer, unsigned *status) {
  constexpr int VPT = ring_vectors(sizeof(T));
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float slots[64];
  auto *head = reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + kRingHead;
  clear_slots(slots, 64);
  ring_init(head, stages);
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  const int group = blockDim.x, t = threadIdx.x, tensors = a.dh != nullptr ? 3 : 2;
  auto copy_y = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.dy) + at.at(a.sdy), a.dim, a.span_y);
  };
  auto copy_h = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.h) + at.at(a.sh), a.dim, a.span_h);
  };
  auto copy_d = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.dh) + at.at(a.sdh), a.dim, a.span_d);
  };
  auto start = [&](int64_t row, int s) {
    const Where at = where(row, a.inner);
    const uint32_t bar = smem_u32(&head->full[s]), buf = smem_u32(ring + s * tensors * buffer);
    const auto cy = copy_y(at), ch = copy_h(at);
    if (tensors == 3) {
      const auto cd = copy_d(at);
      mbar_expect_tx(bar, cy.bytes() + ch.bytes() + cd.bytes());
      copy_start(cd, buf + 2 * buffer, bar);
    } else {
      mbar_expect_tx(bar, cy.bytes() + ch.bytes());
    }
    copy_start(cy, buf, bar);
    copy_start(ch, buf + buffer, bar);
  };
  const int64_t step = gridDim.x;
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < a.rows) start(blockIdx.x + i * step, i);
  float2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  const Weight<AL, T, VPT> w(a.w, a.w32, t, group, a.dim);
  int s = 0, parity = 0;
  uint32_t phase = 0;
  float rstd = blockIdx.x < a.rows ? a.rstd[blockIdx.x] : 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += step) {
    const int t = each_time(int(threadIdx.x));
    const Where at = where(row, a.inner);
    const float next = row + step < a.rows ? a.rstd[row + step] : 0.f;
    ring_wait(head, s, phase, status);
    const uint8_t *buf = ring + s * tensors * buffer;
    Raw8<T> hy[VPT], hh[VPT], hd[VPT];
    take<AL>(hy, copy_y(at), buf, t, group, a.dim);
    take<AL>(hh, copy_h(at), buf + buffer, t, group, a.dim);
    if (tensors == 3) take<AL>(hd, copy_d(at), buf + 2 * buffer, t, group, a.dim);
    row_backward<AL, DROP>(a, now, hy, hh, hd, w, rstd, row, at, t, group, a.dim, slots + 32 * parity, acc);
    parity ^= 1;
    rstd = next;
    // (its barrier came after every thread had read the stage)
    if (*static_cast<volatile int *>(&head->abort_flag)) {
      const int64_t left = (a.rows - row + step - 1) / step;
      if (t == 0) ring_drain(head, s, phase, static_cast<int>(left < stages ? left : stages), stages);
      return;
    }
    if (t == 0 && row + stages * step < a.rows) start(row + stages * step, s);
    if (++s == stages) s = 0, phase ^= 1u;
  }
  if (a.partial == nullptr) return;
  float *out = a.partial + int64_t(blockIdx.x) * a.dim;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<AL>(t, group, j, k);
      if (c < a.dim) out[c] = k & 1 ? acc[j][k / 2].y : acc[j][k / 2].x;
    }
}

// dw = the blocks' sums, added in a fixed order: 32 columns a block, eight
// threads a column.
template <class T>
__global__ void __launch_bounds__(256) k_norm_dw(const float *__restrict__ partial, int blocks,
                                                 int dim, T *__restrict__ dw) {
  __shared__ float part[8][33];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < dim)
    for (int b = slice; b < blocks; b += 8) s += partial[int64_t(b) * dim + c];
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][lane];
    dw[c] = from_f32<T>(s);
  }
}

// How a call runs.
struct Split {
  bool ring;
  int group, vpt, nr, block, per_block;  // threads and vectors of a row; rows at a time
  int stages, blocks_sm;                 // of the ring
  uint32_t buffer;                       // bytes of a row in the ring
};
constexpr int kSms = 152;
constexpr int kRingSmem = 220 * 1024;  // of an SM's, left to its blocks' rings
// Threads of the ring's blocks on an SM: what their registers (80 a thread forward,
// 128 backward) leave room for.
constexpr int kFwdThreads = 768, kBwdThreads = 512;

// Few rows (two an SM at most): as many threads as there are vectors.
bool few_rows(int64_t rows) { return rows <= 2 * kSms; }

// tensors: that are read a row; threads: of an SM.
Split split_of(int dim, int64_t rows, int es, int tensors, int threads_sm) {
  Split s = {};
  const int vectors = (dim + 7) / 8;
  s.nr = 1;
  if (few_rows(rows) && vectors <= 1024) {
    s.vpt = 1;
  } else if (dim > 1024) {
    s.vpt = ring_vectors(es);
    s.group = s.block = ((vectors + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.per_block = 1;
    // (a row may begin and end inside 16 bytes)
    s.buffer = static_cast<uint32_t>((dim * es + 15) / 16 * 16 + 16);
    const int stage = static_cast<int>(s.buffer) * tensors;
    s.blocks_sm = s.block > 512 ? 1 : s.block > 256 ? 1 : threads_sm / s.block;
    if (s.blocks_sm > 8) s.blocks_sm = 8;
    for (; s.blocks_sm > 0; --s.blocks_sm) {
      s.stages = (kRingSmem / s.blocks_sm - 1024 - kRingHead) / stage;
      if (s.stages >= 2) break;
    }
    s.ring = s.blocks_sm > 0 && s.block <= 1024;
    if (s.stages > 4) s.stages = 4;
    if (s.ring) return s;
    s.vpt = 4;
  } else {
    s.vpt = vectors > 64 ? 4 : vectors > 32 ? 2 : 1;
    if (s.vpt == 1) s.nr = 4;
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

// Blocks of the backward, each with a line of partial sums.
int bwd_blocks(const Split &s, int64_t rows) {
  const int64_t n = (rows + s.per_block - 1) / s.per_block;
  const int most = kSms * (s.ring ? s.blocks_sm : 4);
  return static_cast<int>(n < most ? n : most);
}

template <class... P, class A>
cudaError_t launch_ring(void (*kern)(P...), int blocks, const Split &s, int tensors, const A &a,
                        unsigned *status, cudaStream_t st) {
  const size_t smem = kRingHead + size_t(s.stages) * tensors * s.buffer;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(blocks), dim3(s.block), smem, st, a, s.stages, s.buffer, status);
}
template <class T, bool AL, bool DROP, bool FP8>
cudaError_t launch(const FwdArgs &a, const Split &s, int tensors, unsigned *status, cudaStream_t st) {
  if (s.ring) {
    const int64_t most = int64_t(kSms) * s.blocks_sm;
    const int blocks = static_cast<int>(a.rows < most ? a.rows : most);
    auto k = s.block <= 256   ? k_norm_fwd_ring<T, AL, DROP, FP8, 256, kFwdThreads / 256>
             : s.block <= 512 ? k_norm_fwd_ring<T, AL, DROP, FP8, 512, 1>
                              : k_norm_fwd_ring<T, AL, DROP, FP8, 1024, 1>;
    return launch_ring(k, blocks, s, tensors, a, status, st);
  }
  auto k = s.nr == 4    ? k_norm_fwd<T, 1, AL, DROP, FP8, 4, kSmallBlock>
           : s.vpt == 1 ? k_norm_fwd<T, 1, AL, DROP, FP8, 1, 1024>
           : s.vpt == 2 ? k_norm_fwd<T, 2, AL, DROP, FP8, 1, kSmallBlock>
           : s.block <= kSmallBlock ? k_norm_fwd<T, 4, AL, DROP, FP8, 1, kSmallBlock>
                                    : k_norm_fwd<T, 4, AL, DROP, FP8, 1, 1024>;
  const int64_t blocks = (a.rows + s.per_block - 1) / s.per_block;
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(s.block), 0, st, a);
}
template <class T, bool AL, bool DROP>
cudaError_t launch(const BwdArgs &a, const Split &s, int tensors, unsigned *status, cudaStream_t st) {
  const int blocks = bwd_blocks(s, a.rows);
  if (s.ring) {
    auto k = s.block <= 256   ? k_norm_bwd_ring<T, AL, DROP, 256, kBwdThreads / 256>
             : s.block <= 512 ? k_norm_bwd_ring<T, AL, DROP, 512, 1>
                              : k_norm_bwd_ring<T, AL, DROP, 1024, 1>;
    return launch_ring(k, blocks, s, tensors, a, status, st);
  }
  auto k = s.nr == 4    ? k_norm_bwd<T, 1, AL, DROP, 4, kSmallBlock>
           : s.vpt == 1 ? k_norm_bwd<T, 1, AL, DROP, 1, 1024>
           : s.vpt == 2 ? k_norm_bwd<T, 2, AL, DROP, 1, kSmallBlock>
           : s.block <= kSmallBlock ? k_norm_bwd<T, 4, AL, DROP, 1, kSmallBlock>
                                    : k_norm_bwd<T, 4, AL, DROP, 1, 1024>;
  return launch_pdl(k, dim3(blocks), dim3(s.block), 0, st, a);
}
template <class T, bool AL>
cudaError_t launch_any(const FwdArgs &a, const Split &s, int tensors, unsigned *status, cudaStream_t st) {
  if (a.codes != nullptr)
    return a.dropped ? launch<T, AL, true, true>(a, s, tensors, status, st)
                     : launch<T, AL, false, true>(a, s, tensors, status, st);
  return a.dropped ? launch<T, AL, true, false>(a, s, tensors, status, st)
                   : launch<T, AL, false, false>(a, s, tensors, status, st);
}
template <class T, bool AL>
cudaError_t launch_any(const BwdArgs &a, const Split &s, int tensors, unsigned *status, cudaStream_t st) {
  return a.dropped ? launch<T, AL, true>(a, s, tensors, status, st)
                   : launch<T, AL, false>(a, s, tensors, status, st);
}
template <class A>
cudaError_t launch_norm(lora_dtype_t dtype, bool vec, const A &a, const Split &s, int tensors,
                        unsigned *status, cudaStream_t st) {
  if (dtype == LORA_BF16)
    return vec ? launch_any<__nv_bfloat16, true>(a, s, tensors, status, st)
               : launch_any<__nv_bfloat16, false>(a, s, tensors, status, st);
  return vec ? launch_any<float, true>(a, s, tensors, status, st)
             : launch_any<float, false>(a, s, tensors, status, st);
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lora_status_t check_shape(const lora_norm_t *sh, lora_dtype_t dtype) {
  if (sh == nullptr) return fail(LORA_ERR_INVALID_ARG, "shape is NULL");
  if (dtype != LORA_BF16 && dtype != LORA_FP32)
    return fail(LORA_ERR_INVALID_ARG, "dtype %d is not LORA_BF16 or LORA_FP32", int(dtype));
  if (sh->outer < 0 || sh->inner < 0) return fail(LORA_ERR_INVALID_ARG, "outer or inner is negative");
  if (sh->dim < 1) return fail(LORA_ERR_INVALID_ARG, "dim = %d", sh->dim);
  if (sh->dim > kMaxDim) return fail(LORA_ERR_UNSUPPORTED, "dim = %d is over %d", sh->dim, kMaxDim);
  if (sh->inner > 0 && sh->outer > INT_MAX / sh->inner)
    return fail(LORA_ERR_UNSUPPORTED, "2^31 rows or more");
  if (sh->inner > INT_MAX) return fail(LORA_ERR_UNSUPPORTED, "2^31 rows or more");
  if ((sh->weight_fp32 | 1) != 1) return fail(LORA_ERR_INVALID_ARG, "weight_fp32 is 0 or 1");
  if (!(sh->eps >= 0.f) || !(sh->eps < 3e38f))
    return fail(LORA_ERR_INVALID_ARG, "eps = %g is not a number >= 0", sh->eps);
  return LORA_OK;
}

// One tensor of the call: checks it and notes its strides and alignment.
struct Tensors {
  const lora_norm_t *sh;
  int es;
  bool vec;
  lora_status_t add(const void *p, const int64_t *s, const char *name, bool out, Rows &rows,
                    Span *span = nullptr) {
    if (p == nullptr) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, es)) return fail(LORA_ERR_INVALID_ARG, "%s is not aligned to its type", name);
    rows.outer = sh->outer > 1 ? s[0] : 0;
    rows.inner = sh->inner > 1 ? s[1] : 0;
    if (out) {
      const int64_t r0 = rows.outer < 0 ? -rows.outer : rows.outer;
      const int64_t r1 = rows.inner < 0 ? -rows.inner : rows.inner;
      if ((sh->outer > 1 && r0 < sh->dim) || (sh->inner > 1 && r1 < sh->dim))
        return fail(LORA_ERR_INVALID_ARG, "the rows of %s overlap", name);
    }
    vec = vec && aligned(p, 16) && rows.outer % (16 / es) == 0 && rows.inner % (16 / es) == 0;
    if (span != nullptr) {
      int64_t lo = 0, hi = sh->dim;
      for (const int64_t reach : {rows.outer * (sh->outer - 1), rows.inner * (sh->inner - 1)})
        (reach < 0 ? lo : hi) += reach;
      span->first = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(lo * es);
      span->last = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(hi * es);
    }
    return LORA_OK;
  }
};
lora_status_t same_place(const void *out, const Rows &so, const char *out_name, const void *in,
                         const Rows &si, const char *in_name) {
  if (out == in && (so.outer != si.outer || so.inner != si.inner))
    return fail(LORA_ERR_INVALID_ARG, "%s is %s with other strides", out_name, in_name);
  return LORA_OK;
}
lora_status_t check_weight(const void *w, int es, const char *name, bool &vec) {
  if (w == nullptr) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(w, es)) return fail(LORA_ERR_INVALID_ARG, "%s is not aligned to its type", name);
  vec = vec && aligned(w, 16);
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status_t lora_norm_fwd(const lora_norm_t *sh, const void *x, const void *residual,
                            const void *w, const lora_dropout_t *dropout, lora_dtype_t dtype,
                            void *h, void *y, float *rstd, void *codes, float *scale,
                            void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh, dtype));
  FwdArgs a = {};
  LORA_TRY(drop_args(dropout, a.drop));
  if ((codes == nullptr) != (scale == nullptr))
    return fail(LORA_ERR_INVALID_ARG, "codes and scale are given together");
  const int64_t rows = sh->outer * sh->inner;
  if (rows == 0) return LORA_OK;
  a.dropped = dropout != nullptr && a.drop.threshold != 0;
  if (h != nullptr && residual == nullptr && dropout == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "h is x without residual and dropout: give NULL");
  if (y == nullptr && codes == nullptr && h == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "y, codes and h are NULL");
  Tensors ts = {sh, dtype == LORA_BF16 ? 2 : 4, sh->dim % 8 == 0};
  LORA_TRY(ts.add(x, sh->x, "x", false, a.sx, &a.span_x));
  if (residual != nullptr) LORA_TRY(ts.add(residual, sh->residual, "residual", false, a.sr, &a.span_r));
  if (h != nullptr) {
    LORA_TRY(ts.add(h, sh->h, "h", true, a.sh));
    LORA_TRY(same_place(h, a.sh, "h", x, a.sx, "x"));
    LORA_TRY(same_place(h, a.sh, "h", residual, a.sr, "residual"));
  }
  if (y != nullptr) {
    LORA_TRY(ts.add(y, sh->y, "y", true, a.sy));
    LORA_TRY(same_place(y, a.sy, "y", x, a.sx, "x"));
    LORA_TRY(same_place(y, a.sy, "y", residual, a.sr, "residual"));
    if (y == h) return fail(LORA_ERR_INVALID_ARG, "y and h are the same tensor");
  }
  LORA_TRY(check_weight(w, sh->weight_fp32 ? 4 : ts.es, "w", ts.vec));
  if (!aligned(rstd, 4) || !aligned(scale, 4))
    return fail(LORA_ERR_INVALID_ARG, "rstd or scale is not aligned to its type");
  if (codes != nullptr) ts.vec = ts.vec && aligned(codes, 8);
  a.x = x;
  a.res = residual;
  a.w = w;
  // dropout with p = 0 and no residual copies x
  if (h != nullptr && residual == nullptr) a.dropped = 1;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.codes = static_cast<uint8_t *>(codes);
  a.scale = scale;
  a.rows = rows;
  a.inner = static_cast<uint32_t>(sh->inner);
  a.dim = sh->dim;
  a.eps = sh->eps;
  a.w32 = dtype == LORA_FP32 ? 0 : sh->weight_fp32;
  const int tensors = residual != nullptr ? 2 : 1;
  const Split s = split_of(sh->dim, rows, ts.es, tensors, kFwdThreads);
  a.group = s.group;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_NORM, st, "norm",
             [&] { return launch_norm(dtype, ts.vec, a, s, tensors, di.status, st); });
}

size_t lora_norm_workspace_bytes(const lora_norm_t *sh, int with_dw) {
  clear_error();
  if (check_shape(sh, LORA_BF16) != LORA_OK || !with_dw) return 0;
  // (the type, and whether dh is given, move the blocks: room for the most)
  const int64_t rows = sh->outer * sh->inner;
  int most = 0;
  for (int es = 2; es <= 4; es += 2)
    for (int tensors = 2; tensors <= 3; ++tensors) {
      const int n = bwd_blocks(split_of(sh->dim, rows, es, tensors, kBwdThreads), rows);
      most = n > most ? n : most;
    }
  return size_t(most) * sh->dim * sizeof(float);
}

lora_status_t lora_norm_bwd(const lora_norm_t *sh, const void *dy, const void *h, const void *w,
                            const float *rstd, const void *dh, const lora_dropout_t *dropout,
                            lora_dtype_t dtype, void *dx, void *dresidual, void *dw,
                            void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  LORA_TRY(check_shape(sh, dtype));
  BwdArgs a = {};
  LORA_TRY(drop_args(dropout, a.drop));
  const int64_t rows = sh->outer * sh->inner;
  const int ws_es = sh->weight_fp32 || dtype == LORA_FP32 ? 4 : 2;
  if (dw != nullptr && !aligned(dw, ws_es))
    return fail(LORA_ERR_INVALID_ARG, "dw is not aligned to its type");
  const int tensors = dh != nullptr ? 3 : 2;
  const Split s = split_of(sh->dim, rows, dtype == LORA_BF16 ? 2 : 4, tensors, kBwdThreads);
  const int blocks = bwd_blocks(s, rows);
  bool vec = sh->dim % 8 == 0;
  if (rows > 0) {
    Tensors ts = {sh, dtype == LORA_BF16 ? 2 : 4, vec};
    LORA_TRY(ts.add(dy, sh->dy, "dy", false, a.sdy, &a.span_y));
    LORA_TRY(ts.add(h, sh->h, "h", false, a.sh, &a.span_h));
    if (dh != nullptr) LORA_TRY(ts.add(dh, sh->dh, "dh", false, a.sdh, &a.span_d));
    LORA_TRY(ts.add(dx, sh->dx, "dx", true, a.sdx));
    LORA_TRY(same_place(dx, a.sdx, "dx", dy, a.sdy, "dy"));
    LORA_TRY(same_place(dx, a.sdx, "dx", dh, a.sdh, "dh"));
    LORA_TRY(same_place(dx, a.sdx, "dx", h, a.sh, "h"));
    if (dresidual != nullptr) {
      LORA_TRY(ts.add(dresidual, sh->dresidual, "dresidual", true, a.sdr));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", dy, a.sdy, "dy"));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", dh, a.sdh, "dh"));
      LORA_TRY(same_place(dresidual, a.sdr, "dresidual", h, a.sh, "h"));
      if (dresidual == dx) return fail(LORA_ERR_INVALID_ARG, "dx and dresidual are the same tensor");
    }
    LORA_TRY(check_weight(w, ws_es, "w", ts.vec));
    if (rstd == nullptr || !aligned(rstd, 4))
      return fail(LORA_ERR_INVALID_ARG, "rstd is NULL or not aligned");
    vec = ts.vec;
  }
  if (dw != nullptr)
    LORA_TRY(check_ws(workspace, workspace_bytes, size_t(blocks) * sh->dim * sizeof(float)));
  if (rows == 0 && dw == nullptr) return LORA_OK;
  a.dropped = dropout != nullptr && a.drop.threshold != 0;
  a.dy = dy;
  a.h = h;
  a.w = w;
  a.dh = dh;
  a.rstd = rstd;
  a.dx = dx;
  a.dres = dresidual;
  a.partial = dw != nullptr ? static_cast<float *>(workspace) : nullptr;
  a.rows = rows;
  a.inner = static_cast<uint32_t>(sh->inner);
  a.dim = sh->dim;
  a.w32 = dtype == LORA_FP32 ? 0 : sh->weight_fp32;
  a.group = s.group;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows > 0)
    LORA_TRY(run(LORA_K_NORM_BWD, st, "norm backward",
                 [&] { return launch_norm(dtype, vec, a, s, tensors, di.status, st); }));
  if (dw == nullptr) return LORA_OK;
  return run(LORA_K_NORM_BWD, st, "norm dw", [&] {
    const dim3 grid((sh->dim + 31) / 32);
    const float *partial = static_cast<const float *>(workspace);
    return ws_es == 4
               ? launch_pdl(k_norm_dw<float>, grid, dim3(256), 0, st, partial, blocks, int(sh->dim),
                            static_cast<float *>(dw))
               : launch_pdl(k_norm_dw<__nv_bfloat16>, grid, dim3(256), 0, st, partial, blocks,
                            int(sh->dim), static_cast<__nv_bfloat16 *>(dw));
  });
}

}  // extern "C"
