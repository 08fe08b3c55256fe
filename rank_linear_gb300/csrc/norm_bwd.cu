// norm_bwd.cu -- the norm's backward kernels (include/lora_norm.h).
#include "norm.cuh"

namespace lora {
namespace {

// ---- backward ----
// What a row's threads do with it: g = dy w and h r, their mean product, then
// d = r (g - h r mean) + dh, dropped out where the branch was.
template <int AL, bool KEEP, class T, int VPT>
__device__ __forceinline__ void row_backward(const NormBwdArgs &a, const DropNow &now,
                                             const Raw8<T> (&hy)[VPT], const Raw8<T> (&hh)[VPT],
                                             const Raw8<T> (&hd)[VPT], const Weight<AL, KEEP, T, VPT> &w,
                                             float rstd, bool drop, int64_t row, const Where &at, int t,
                                             int group, int dim, float *slot, float2 (&acc)[VPT][4], int m = 0,
                                             const uint32_t *own = nullptr) {
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
  const float along = over_group<false>(s.x + s.y, group, slot) * a.inv_dim;
  // d = r (g - h r mean) + dh: the square of r alone would leave fp32 where h r does not
  const float2 back = both(-along);
  rstd = each_time(rstd);  // (h r is made again: held since the sum, it spilled)
  T *dx = static_cast<T *>(a.dx) + at.at(a.sdx);
  T *dres = static_cast<T *>(a.dres) + at.at(a.sdr);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 d[4], u[4];
    w.get(j, t, group, a.dim, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 hat = mul2(hh[j].pair(i), both(rstd));
      d[i] = fma2(hat, back, mul2(hy[j].pair(i), u[i]));
      d[i] = a.dh != nullptr ? fma2(d[i], both(rstd), hd[j].pair(i)) : mul2(d[i], both(rstd));
    }
    if (a.dres != nullptr) put<AL>(dres, d, t, group, j, dim, m, AL == kShifted ? own[j] : 255u);
    if (drop) drop_vector<AL>(a.drop, now, row, t, group, j, d);
    put<AL>(dx, d, t, group, j, dim, m, AL == kShifted ? own[j] : 255u);
  }
}

// Straight into registers: blocks stay and take NR rows a group at a time; each
// thread adds up dy h r of its columns over the rows that it took.
template <class T, int VPT, int AL, int NR, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_bwd(const __grid_constant__ NormBwdArgs a) {
  __shared__ __align__(16) float slots[64];
  __shared__ float cols[kSmallBlock * VPT * 8];  // dw of the groups of a small block
  clear_slots(slots, 64);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  const int group = a.group;
  const int t = threadIdx.x % group, sub = threadIdx.x / group, subs = blockDim.x / group;
  float2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  const Weight<AL, true, T, VPT> w(a.w, a.w32, t, group, a.dim);
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
      row_backward<AL, true>(a, now, hy[n], hh[n], hd[n], w, rstd[n], a.dropped != 0, row,
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
template <class T, int AL, bool DROP, int MAX, int BLOCKS>
__global__ void __launch_bounds__(MAX, BLOCKS)
    k_norm_bwd_ring(const __grid_constant__ NormBwdArgs a, int stages, uint32_t buffer, unsigned *status) {
  constexpr int VPT = kRingVectors;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float slots[64];
  auto *head = reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + kRingHead;
  clear_slots(slots, 64);
  ring_init(head, stages);
  griddep_wait();
  fence_proxy_async_global();  // what the kernels before wrote, for this thread's copies
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
  ShiftCopy shift = {};
  if constexpr (AL == kShifted)
    shift = ShiftCopy::of(static_cast<const T *>(a.dy) + int64_t(blockIdx.x) * a.sdy.outer, a.dim, a.rows);
  auto start = [&](int64_t row, int s) {
    const Where at = where(row, a.inner);
    const uint32_t bar = smem_u32(&head->full[s]), buf = smem_u32(ring + s * tensors * buffer);
    if constexpr (AL == kShifted) {
      const T *y = static_cast<const T *>(a.dy) + at.at(a.sdy), *h = static_cast<const T *>(a.h) + at.at(a.sh);
      const T *d = static_cast<const T *>(a.dh) + at.at(a.sdh);
      mbar_expect_tx(bar, copy_bytes(shift, y, row, a.dim, a.span_y) + copy_bytes(shift, h, row, a.dim, a.span_h) +
                              (tensors == 3 ? copy_bytes(shift, d, row, a.dim, a.span_d) : 0u));
      copy_start(shift, y, row, a.dim, a.span_y, buf, bar);
      copy_start(shift, h, row, a.dim, a.span_h, buf + buffer, bar);
      if (tensors == 3) copy_start(shift, d, row, a.dim, a.span_d, buf + 2 * buffer, bar);
      return;
    }
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
  // (the thread that starts the copies: of a warp without a shifted row's ends)
  const int starter = AL == kShifted ? group / 64 * 32 : 0;
  if (t == starter)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < a.rows) start(blockIdx.x + i * step, i);
  float2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  uint32_t own[VPT] = {};
  if constexpr (AL == kShifted) own_bits(own, t, group, a.dim, shift.m);
  const Weight<AL, true, T, VPT> w(a.w, a.w32, t, group, a.dim, shift.m);
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
    if constexpr (AL == kShifted) {
      take(hy, shift, static_cast<const T *>(a.dy) + at.at(a.sdy), row, a.span_y, buf, t, group, a.dim);
      take(hh, shift, static_cast<const T *>(a.h) + at.at(a.sh), row, a.span_h, buf + buffer, t, group, a.dim);
      if (tensors == 3)
        take(hd, shift, static_cast<const T *>(a.dh) + at.at(a.sdh), row, a.span_d, buf + 2 * buffer, t, group, a.dim);
      if (!all_own(own)) {
        only_own(hy, own);
        only_own(hh, own);
      }
    } else {
      take<AL>(hy, copy_y(at), buf, t, group, a.dim);
      take<AL>(hh, copy_h(at), buf + buffer, t, group, a.dim);
      if (tensors == 3) take<AL>(hd, copy_d(at), buf + 2 * buffer, t, group, a.dim);
    }
    row_backward<AL, true>(a, now, hy, hh, hd, w, rstd, DROP, row, at, t, group, a.dim, slots + 32 * parity, acc, shift.m,
                           own);
    parity ^= 1;
    rstd = next;
    // (its barrier came after every thread had read the stage)
    if (*static_cast<volatile int *>(&head->abort_flag)) {
      const int64_t left = (a.rows - row + step - 1) / step;
      if (t == 0) ring_drain(head, s, phase, static_cast<int>(left < stages ? left : stages), stages);
      return;
    }
    if (t == starter && row + stages * step < a.rows) start(row + stages * step, s);
    if (++s == stages) s = 0, phase ^= 1u;
  }
  if (a.partial == nullptr) return;
  float *out = a.partial + int64_t(blockIdx.x) * a.dim;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<AL>(t, group, j, k) - shift.m;
      if (c >= 0 && c < a.dim) out[c] = k & 1 ? acc[j][k / 2].y : acc[j][k / 2].x;
    }
}

// Narrow rows that lie side by side (the heads of a token), over the ring: its row is
// `inner` of them, each of which belongs to `lanes` neighbouring threads of a warp.
template <class T, int VPT, bool DROP>
__global__ void __launch_bounds__(heads_threads(VPT) / 2, 2)
    k_norm_bwd_heads(const __grid_constant__ NormBwdArgs a, int stages, uint32_t buffer,
                     unsigned *status) {
  extern __shared__ __align__(128) uint8_t smem[];
  auto *head = reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + kRingHead;
  ring_init(head, stages);
  griddep_wait();
  fence_proxy_async_global();  // what the kernels before wrote, for this thread's copies
  griddep_launch_dependents();
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  const int lanes = a.group, tl = threadIdx.x % lanes, sub = threadIdx.x / lanes;
  const int tensors = a.dh != nullptr ? 3 : 2;
  const int inner = static_cast<int>(a.inner.n), wide = inner * a.dim;
  const int64_t entries = a.rows / inner, step = gridDim.x;
  auto start = [&](int64_t o, int s) {
    const uint32_t bar = smem_u32(&head->full[s]), buf = smem_u32(ring + s * tensors * buffer);
    const uint32_t n = static_cast<uint32_t>(wide) * static_cast<uint32_t>(sizeof(T));
    mbar_expect_tx(bar, n * tensors);
    bulk_load(buf, static_cast<const T *>(a.dy) + o * a.sdy.outer, n, bar);
    bulk_load(buf + buffer, static_cast<const T *>(a.h) + o * a.sh.outer, n, bar);
    if (tensors == 3) bulk_load(buf + 2 * buffer, static_cast<const T *>(a.dh) + o * a.sdh.outer, n, bar);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < entries) start(blockIdx.x + i * step, i);
  float2 acc[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  const Weight<kAligned, true, T, VPT> w(a.w, a.w32, tl, lanes, a.dim);
  const int dim = sub < inner ? a.dim : 0;
  int s = 0;
  uint32_t phase = 0;
  float rstd = sub < inner && blockIdx.x < entries ? a.rstd[int64_t(blockIdx.x) * inner + sub] : 0.f;
  for (int64_t o = blockIdx.x; o < entries; o += step) {
    const int t = each_time(tl);
    const float next = sub < inner && o + step < entries ? a.rstd[(o + step) * inner + sub] : 0.f;
    Raw8<T> hy[VPT], hh[VPT], hd[VPT];
    ring_wait(head, s, phase, status);
    const T *buf = reinterpret_cast<const T *>(ring + s * tensors * buffer) + sub * a.dim;
    const T *buf_h = reinterpret_cast<const T *>(ring + (s * tensors + 1) * buffer) + sub * a.dim;
    fetch<kAligned>(hy, buf, t, lanes, dim);
    fetch<kAligned>(hh, buf_h, t, lanes, dim);
    if (tensors == 3)
      fetch<kAligned>(hd, reinterpret_cast<const T *>(ring + (s * tensors + 2) * buffer) + sub * a.dim, t, lanes, dim);
    __syncthreads();  // every thread has read the stage
    if (*static_cast<volatile int *>(&head->abort_flag)) {
      const int64_t left = (entries - o + step - 1) / step;
      if (threadIdx.x == 0) ring_drain(head, s, phase, static_cast<int>(left < stages ? left : stages), stages);
      return;
    }
    if (threadIdx.x == 0 && o + stages * step < entries) start(o + stages * step, s);
    if (++s == stages) s = 0, phase ^= 1u;
    row_backward<kAligned, true>(a, now, hy, hh, hd, w, rstd, DROP, o * inner + sub, Where{o, sub}, t, lanes, dim,
                                 nullptr, acc);
    rstd = next;
  }
  if (a.partial == nullptr) return;
  // the sums of the threads with the same columns, in their order; the ring is free
  float *cols = reinterpret_cast<float *>(ring);
  const int groups = blockDim.x / lanes;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<kAligned>(tl, lanes, j, k);
      if (c < a.dim) cols[sub * a.dim + c] = k & 1 ? acc[j][k / 2].y : acc[j][k / 2].x;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
    float sum = 0.f;
    for (int i = 0; i < groups; ++i) sum += cols[i * a.dim + c];
    a.partial[int64_t(blockIdx.x) * a.dim + c] = sum;
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
  if (c < dim) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += 8) s += partial[int64_t(b) * dim + c];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][lane];
    dw[c] = from_f32<T>(s);
  }
}

template <class T, int AL, bool DROP>
cudaError_t launch_bwd_ring(const NormBwdArgs &a, const NormSplit &s, int tensors, unsigned *status,
                            cudaStream_t st) {
  constexpr int ES = sizeof(T), MID = AL == kAligned || (AL == kShifted && ES == 2) ? 384 : 320;
  static std::atomic<uint64_t> allowed[3];
  const int which = s.block <= 256 ? 0 : s.block <= MID ? 1 : 2;
  auto k = which == 0   ? k_norm_bwd_ring<T, AL, DROP, 256, ring_blocks(256, AL, ES)>
           : which == 1 ? k_norm_bwd_ring<T, AL, DROP, MID, ring_blocks(MID, AL, ES)>
                        : k_norm_bwd_ring<T, AL, DROP, 512, 1>;
  return launch_ring(k, allowed[which], norm_bwd_blocks(s, a.rows), s, tensors, a, status, st);
}
template <class T, bool DROP>
cudaError_t launch_bwd_heads(const NormBwdArgs &a, const NormSplit &s, int tensors, unsigned *status,
                             cudaStream_t st) {
  static std::atomic<uint64_t> allowed[2];
  const int which = s.vpt == 3;
  auto k = which ? k_norm_bwd_heads<T, 3, DROP> : k_norm_bwd_heads<T, 2, DROP>;
  return launch_ring(k, allowed[which], norm_bwd_blocks(s, a.rows / a.inner.n), s, tensors, a, status, st);
}
template <class T, int AL>
cudaError_t launch_any(const NormBwdArgs &a, const NormSplit &s, int tensors, unsigned *status, cudaStream_t st) {
  if (s.heads)
    return a.dropped ? launch_bwd_heads<T, true>(a, s, tensors, status, st)
                     : launch_bwd_heads<T, false>(a, s, tensors, status, st);
  if (s.shifted) {
    if constexpr (AL == kLoose) return launch_bwd_ring<T, kShifted, false>(a, s, tensors, status, st);
  }
  if (s.ring)
    return a.dropped ? launch_bwd_ring<T, AL, true>(a, s, tensors, status, st)
                     : launch_bwd_ring<T, AL, false>(a, s, tensors, status, st);
  constexpr int NR = narrow_rows(AL != kLoose);
  auto k = s.nr == NR   ? k_norm_bwd<T, 1, AL, NR, kSmallBlock>
           : s.vpt == 1 ? k_norm_bwd<T, 1, AL, 1, 1024>
           : s.block <= kSmallBlock ? k_norm_bwd<T, 4, AL, 1, kSmallBlock>
                                    : k_norm_bwd<T, 4, AL, 1, 1024>;
  if constexpr (AL == kAligned)
    if (s.vpt == 3) k = k_norm_bwd<T, 3, AL, 1, kSmallBlock>;  // (96 vectors at most)
  return launch_pdl(k, dim3(norm_bwd_blocks(s, a.rows)), dim3(s.block), 0, st, a);
}
}  // namespace

cudaError_t launch_norm_bwd(lora_dtype_t dtype, bool vec, const NormBwdArgs &a, const NormSplit &s, int tensors,
                            unsigned *status, cudaStream_t st) {
  if (dtype == LORA_BF16)
    return vec ? launch_any<__nv_bfloat16, true>(a, s, tensors, status, st)
               : launch_any<__nv_bfloat16, false>(a, s, tensors, status, st);
  return vec ? launch_any<float, true>(a, s, tensors, status, st)
             : launch_any<float, false>(a, s, tensors, status, st);
}

cudaError_t launch_norm_dw(bool fp32, const float *partial, int blocks, int dim, void *dw,
                           cudaStream_t st) {
  const dim3 grid((dim + 31) / 32);
  return fp32 ? launch_pdl(k_norm_dw<float>, grid, dim3(256), 0, st, partial, blocks, dim,
                           static_cast<float *>(dw))
              : launch_pdl(k_norm_dw<__nv_bfloat16>, grid, dim3(256), 0, st, partial, blocks, dim,
                           static_cast<__nv_bfloat16 *>(dw));
}

}  // namespace lora
