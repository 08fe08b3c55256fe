// norm_fwd.cu -- the norm's forward kernels (include/lora_norm.h).
#include "e4m3.cuh"
#include "norm.cuh"

namespace lora {
namespace {

// r = (ss / dim + eps)^(-1/2) of the row in v.  Where the squares leave the
// range of fp32, or are so small that they lose bits and eps does not cover it (a
// square rounds by 2^-150 at most), the sum is taken again of values scaled by 2^-100
// or 2^100 (exact; 32768 squares of 2^128 2^-100 stay below 2^71, and the scaled
// sum of a row whose mean square is below 2^-100 below 2^115), which the result is
// scaled by as well.
template <class T, int VPT>
__device__ __forceinline__ float rstd_of(const Raw8<T> (&v)[VPT], float inv_dim, float eps, int group,
                                         float *slot, float *slot2) {
  float2 s = both(0.f);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(v[j].pair(i), v[j].pair(i), s);
  const float ss = over_group<false>(s.x + s.y, group, slot), mean = fmaf(ss, inv_dim, eps);
  // the same in every thread of a block-wide group; the smaller groups of a
  // warp shuffle together
  const bool near = mean < 0x1p-100f, far = near || !(ss <= 1e38f);
  if (!(group > 32 ? far : __any_sync(0xffffffffu, far))) return rsqrtf(mean);
  const float by = near ? 0x1p100f : 0x1p-100f;
  float s2 = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = mul2(v[j].pair(i), both(by));
      s2 = fmaf(u.x, u.x, fmaf(u.y, u.y, s2));
    }
  s2 = over_group<false>(s2, group, slot2);
  return far ? by * rsqrtf(fmaf(s2, inv_dim, eps * by * by)) : rsqrtf(mean);
}

// x becomes drop(x) + residual, as the stream holds it (rounded once to the
// dtype: the norm is of that), written to h.
template <int AL, class T, int VPT>
__device__ __forceinline__ void to_stream(const NormFwdArgs &a, const DropNow &now, Raw8<T> (&x)[VPT],
                                          const Raw8<T> (&res)[VPT], bool drop, int64_t row, T *h,
                                          int t, int group, int dim, int m = 0,
                                          const uint32_t *own = nullptr) {
  if (!drop && a.res == nullptr) return;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[j].pair(i);
    if (drop) drop_vector<AL>(a.drop, now, row, t, group, j, v);
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], res[j].pair(i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j].set(i, v[i]);
    if (a.h != nullptr) put<AL>(h, x[j], t, group, j, dim, m, AL == kShifted ? own[j] : 255u);
    if (AL == kAligned && (t + j * group) * 8 >= dim) {  // (a mask of zeros may have set a sign)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j].set(i, both(0.f));
    }
  }
}

// y = h r w to memory, and the codes and the scale.
template <int AL, bool FP8, class T, int VPT>
__device__ __forceinline__ void to_outputs(const NormFwdArgs &a, const Raw8<T> (&h)[VPT],
                                           const Weight<AL, true, T, VPT> &w, float rstd, int64_t row, T *y,
                                           int t, int group, int dim, float *slot, int m = 0,
                                           const uint32_t *own = nullptr) {
  float2 v[FP8 ? VPT : 1][4];
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float2 u[4], (&o)[4] = v[FP8 ? j : 0];
    w.get(j, t, group, a.dim, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = mul2(mul2(h[j].pair(i), both(rstd)), u[i]);
    }
    if (FP8 && a.codes != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(o[i].x), fabsf(o[i].y)));
    }
    if (a.y != nullptr) put<AL>(y, o, t, group, j, dim, m, AL == kShifted ? own[j] : 255u);
  }
  if (FP8 && a.codes != nullptr) {
    top = over_group<true>(top, group, slot);
    // an infinite row's scale is that of the largest finite number
    const int e = top <= 3.4028234e38f ? max(pow2_exponent(top), -126) : 120;
    const float inv = ldexpf(1.f, -e);
    if (dim > 0 && t == 0) a.scale[row] = ldexpf(1.f, e);
    uint8_t *q = a.codes + row * a.dim;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if constexpr (AL != kLoose) {
        const int c = (t + j * group) * 8 - m;
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = to_e4m3x2(mul2(v[j][i], both(inv)));
        if (AL == kAligned ? c < dim : own[j] == 255u) {
          *reinterpret_cast<uint2 *>(q + c) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
        } else if (AL == kShifted) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (own[j] >> k & 1u) q[c + k] = static_cast<uint8_t>(p[k / 2] >> 8 * (k % 2));
        }
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

// Forward, straight into registers: blocks stay and take NR rows a group of threads
// at a time, all of them on their way at once.
template <class T, int VPT, int AL, int NR, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_fwd(const __grid_constant__ NormFwdArgs a) {
  __shared__ __align__(16) float slots[192];  // of a round, and of the next
  clear_slots(slots, 192);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int group = a.group;
  const int sub = threadIdx.x / group, subs = blockDim.x / group;
  const DropNow now = drop_now(a.drop);
  const Weight<AL, true, T, VPT> w(a.w, a.w32, threadIdx.x % group, group, a.dim);
  float *slot = slots;
  const int64_t step = int64_t(gridDim.x) * subs * NR;
  for (int64_t first = int64_t(blockIdx.x) * subs * NR; first < a.rows; first += step) {
    const int t = each_time(int(threadIdx.x % group));
    Raw8<T> hx[NR][VPT], hr[NR][VPT];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int64_t row = first + n * subs + sub;
      const int dim = row < a.rows ? a.dim : 0;  // a group without a row holds zeros
      const Where at = where(row < a.rows ? row : 0, a.inner);
      fetch<AL>(hx[n], static_cast<const T *>(a.x) + at.at(a.sx), t, group, dim);
      if (a.res != nullptr) fetch<AL>(hr[n], static_cast<const T *>(a.res) + at.at(a.sr), t, group, dim);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int64_t row = first + n * subs + sub;
      const bool live = row < a.rows;
      const int dim = live ? a.dim : 0;
      const Where at = where(live ? row : 0, a.inner);
      to_stream<AL>(a, now, hx[n], hr[n], a.dropped != 0, row, static_cast<T *>(a.h) + at.at(a.sh), t,
                    group, dim);
      const float rstd = rstd_of(hx[n], a.inv_dim, a.eps, group, slot, slot + 32);
      if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
      to_outputs<AL, true>(a, hx[n], w, rstd, row, static_cast<T *>(a.y) + at.at(a.sy), t, group, dim,
                           slot + 64);
      slot = slot == slots ? slots + 96 : slots;
    }
  }
}

// Forward over the ring: block b takes rows b, b + grid, ...
template <class T, int AL, bool DROP, bool FP8, int MAX, int BLOCKS>
__global__ void __launch_bounds__(MAX, BLOCKS)
    k_norm_fwd_ring(const __grid_constant__ NormFwdArgs a, int stages, uint32_t buffer, unsigned *status) {
  constexpr int VPT = kRingVectors;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float slots[128];
  auto *head = reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + kRingHead;
  clear_slots(slots, 128);
  ring_init(head, stages);
  griddep_wait();
  fence_proxy_async_global();  // what the kernels before wrote, for this thread's copies
  griddep_launch_dependents();
  const DropNow now = DROP ? drop_now(a.drop) : DropNow{};
  const int group = blockDim.x, t = threadIdx.x, tensors = a.res != nullptr ? 2 : 1;
  auto copy_x = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.x) + at.at(a.sx), a.dim, a.span_x);
  };
  auto copy_r = [&](const Where &at) {
    return row_copy<AL>(static_cast<const T *>(a.res) + at.at(a.sr), a.dim, a.span_r);
  };
  ShiftCopy shift = {};
  if constexpr (AL == kShifted)
    shift = ShiftCopy::of(static_cast<const T *>(a.x) + int64_t(blockIdx.x) * a.sx.outer, a.dim, a.rows);
  auto start = [&](int64_t row, int s) {
    const Where at = where(row, a.inner);
    const uint32_t bar = smem_u32(&head->full[s]), buf = smem_u32(ring + s * tensors * buffer);
    if constexpr (AL == kShifted) {
      const T *x = static_cast<const T *>(a.x) + at.at(a.sx), *r = static_cast<const T *>(a.res) + at.at(a.sr);
      mbar_expect_tx(bar, copy_bytes(shift, x, row, a.dim, a.span_x) +
                              (tensors == 2 ? copy_bytes(shift, r, row, a.dim, a.span_r) : 0u));
      copy_start(shift, x, row, a.dim, a.span_x, buf, bar);
      if (tensors == 2) copy_start(shift, r, row, a.dim, a.span_r, buf + buffer, bar);
      return;
    }
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
  // (the thread that starts the copies: of a warp without a shifted row's ends)
  const int starter = AL == kShifted ? group / 64 * 32 : 0;
  if (t == starter)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < a.rows) start(blockIdx.x + i * step, i);
  uint32_t own[VPT] = {};
  if constexpr (AL == kShifted) own_bits(own, t, group, a.dim, shift.m);
  const Weight<AL, true, T, VPT> w(a.w, a.w32, t, group, a.dim, shift.m);
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
      if constexpr (AL == kShifted) {
        take(x, shift, static_cast<const T *>(a.x) + at.at(a.sx), row, a.span_x, buf, t, group, a.dim);
        if (tensors == 2)
          take(r, shift, static_cast<const T *>(a.res) + at.at(a.sr), row, a.span_r, buf + buffer, t, group, a.dim);
        if (!all_own(own)) {
          only_own(x, own);
          if (tensors == 2) only_own(r, own);
        }
      } else {
        take<AL>(x, copy_x(at), buf, t, group, a.dim);
        if (tensors == 2) take<AL>(r, copy_r(at), buf + buffer, t, group, a.dim);
      }
      to_stream<AL>(a, now, x, r, DROP, row, static_cast<T *>(a.h) + at.at(a.sh), t, group, a.dim, shift.m,
                    own);
    }
    // its barrier: every thread has read the stage
    const float rstd = rstd_of(x, a.inv_dim, a.eps, group, slots + 32 * parity, slots + 64);
    parity ^= 1;
    if (*static_cast<volatile int *>(&head->abort_flag)) {  // a copy that never came
      const int64_t left = (a.rows - row + step - 1) / step;
      if (t == 0) ring_drain(head, s, phase, static_cast<int>(left < stages ? left : stages), stages);
      return;
    }
    if (t == starter) {
      if (row + stages * step < a.rows) start(row + stages * step, s);
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if (++s == stages) s = 0, phase ^= 1u;
    to_outputs<AL, FP8>(a, x, w, rstd, row, static_cast<T *>(a.y) + at.at(a.sy), t, group, a.dim,
                        slots + 96, shift.m, own);
  }
}

template <class T, int AL, bool DROP, bool FP8>
cudaError_t launch_fwd_ring(const NormFwdArgs &a, const NormSplit &s, int tensors, unsigned *status,
                            cudaStream_t st) {
  const int64_t most = int64_t(kSms) * s.blocks_sm;
  const int blocks = static_cast<int>(a.rows < most ? a.rows : most);
  constexpr int ES = sizeof(T), MID = AL == kAligned || (AL == kShifted && ES == 2) ? 384 : 320;
  static std::atomic<uint64_t> allowed[3];
  const int which = s.block <= 256 ? 0 : s.block <= MID ? 1 : 2;
  auto k = which == 0   ? k_norm_fwd_ring<T, AL, DROP, FP8, 256, ring_blocks(256, AL, ES)>
           : which == 1 ? k_norm_fwd_ring<T, AL, DROP, FP8, MID, ring_blocks(MID, AL, ES)>
                        : k_norm_fwd_ring<T, AL, DROP, FP8, 512, 1>;
  return launch_ring(k, allowed[which], blocks, s, tensors, a, status, st);
}
template <class T, int AL>
cudaError_t launch_any(const NormFwdArgs &a, const NormSplit &s, int tensors, unsigned *status, cudaStream_t st) {
  if (s.shifted) {
    if constexpr (AL == kLoose) {
      if constexpr (sizeof(T) == 2)
        if (a.codes != nullptr) return launch_fwd_ring<T, kShifted, false, true>(a, s, tensors, status, st);
      return launch_fwd_ring<T, kShifted, false, false>(a, s, tensors, status, st);
    }
  }
  if (s.ring) {
    if constexpr (sizeof(T) == 2) {
      if (a.codes != nullptr)
        return a.dropped ? launch_fwd_ring<T, AL, true, true>(a, s, tensors, status, st)
                         : launch_fwd_ring<T, AL, false, true>(a, s, tensors, status, st);
    }
    return a.dropped ? launch_fwd_ring<T, AL, true, false>(a, s, tensors, status, st)
                     : launch_fwd_ring<T, AL, false, false>(a, s, tensors, status, st);
  }
  constexpr int NR = narrow_rows(AL != kLoose);
  auto k = s.nr == NR   ? k_norm_fwd<T, 1, AL, NR, kSmallBlock>
           : s.vpt == 1 ? k_norm_fwd<T, 1, AL, 1, 1024>
           : s.block <= kSmallBlock ? k_norm_fwd<T, 4, AL, 1, kSmallBlock>
                                    : k_norm_fwd<T, 4, AL, 1, 1024>;
  if constexpr (AL == kAligned)
    if (s.vpt == 3) k = k_norm_fwd<T, 3, AL, 1, kSmallBlock>;  // (96 vectors at most)
  // (blocks stay: 12 of 128 threads an SM, or two wider ones, at most)
  const int64_t want = (a.rows + s.per_block - 1) / s.per_block;
  const int64_t most = int64_t(kSms) * (s.block <= kSmallBlock ? 12 : 2);
  return launch_pdl(k, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(s.block), 0, st, a);
}
}  // namespace

cudaError_t launch_norm_fwd(lora_dtype_t dtype, bool vec, const NormFwdArgs &a, const NormSplit &s, int tensors,
                            unsigned *status, cudaStream_t st) {
  if (dtype == LORA_BF16)
    return vec ? launch_any<__nv_bfloat16, true>(a, s, tensors, status, st)
               : launch_any<__nv_bfloat16, false>(a, s, tensors, status, st);
  return vec ? launch_any<float, true>(a, s, tensors, status, st)
             : launch_any<float, false>(a, s, tensors, status, st);
}

}  // namespace lora
