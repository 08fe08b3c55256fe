// norm.cu -- root-mean-square norm with the residual's addition, dropout of the
// branch and an 8-bit output (include/lora_norm.h; ch05 "Acceleration
// principles: Triton kernels and fused LoRA", §5.4: one pass over the row).
//
// A row stays in the registers of the threads that read it: it is read once,
// its sum of squares (and largest magnitude) go through shuffles and shared
// memory, and it is written once.
#include <climits>

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

struct FwdArgs {
  const void *x, *res, *w;
  void *h, *y;
  float *rstd, *scale;
  uint8_t *codes;
  Rows sx, sr, sh, sy;
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

// Elements of vector j of thread t of a row's `group` threads.  Aligned rows:
// eight that lie side by side (vector t + j group).  Others: eight that lie
// `group` apart, so that a warp's loads cover neighbours.
template <bool AL>
__device__ __forceinline__ int element(int t, int group, int j, int k) {
  return AL ? (t + j * group) * 8 + k : (j * 8 + k) * group + t;
}

template <bool AL, class T>
struct Held;  // a vector as loaded
template <class T>
struct Held<true, T> {
  Raw8<T> r;
};
template <class T>
struct Held<false, T> {
  T e[8];
};

template <class T>
__device__ __forceinline__ void fetch(Held<true, T> &o, const T *p, int t, int group, int j, int dim) {
  const int c = (t + j * group) * 8;
  if (c < dim) load_raw(p + c, o.r);
}
template <class T>
__device__ __forceinline__ void fetch(Held<false, T> &o, const T *p, int t, int group, int j, int dim) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = element<false>(t, group, j, k);
    if (c < dim) o.e[k] = p[c];
  }
}
// ... as fp32, zero past the row's end.
template <class T>
__device__ __forceinline__ void open(const Held<true, T> &o, int t, int group, int j, int dim,
                                     float (&v)[8]) {
  unpack(o.r, v);
  if ((t + j * group) * 8 >= dim) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
  }
}
template <class T>
__device__ __forceinline__ void open(const Held<false, T> &o, int t, int group, int j, int dim,
                                     float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = element<false>(t, group, j, k) < dim ? to_f32(o.e[k]) : 0.f;
}
template <bool AL, class T>
__device__ __forceinline__ void put(T *p, int t, int group, int j, int dim, const float (&v)[8]) {
  if constexpr (AL) {
    const int c = (t + j * group) * 8;
    if (c < dim) store8(p + c, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = element<false>(t, group, j, k);
      if (c < dim) p[c] = from_f32<T>(v[k]);
    }
  }
}
// The weight's vector, of its own type.
template <bool AL, class T>
__device__ __forceinline__ void weight(const void *w, int w32, int t, int group, int j, int dim,
                                       float (&v)[8]) {
  if (w32) {
    Held<AL, float> o;
    fetch(o, static_cast<const float *>(w), t, group, j, dim);
    open(o, t, group, j, dim, v);
  } else {
    Held<AL, T> o;
    fetch(o, static_cast<const T *>(w), t, group, j, dim);
    open(o, t, group, j, dim, v);
  }
}
template <bool AL>
__device__ __forceinline__ void drop_vector(const DropArgs &d, int64_t row, int t, int group, int j,
                                            float (&v)[8]) {
  if constexpr (AL) {
    drop8(d, static_cast<uint32_t>(t + j * group), row, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = static_cast<uint32_t>(element<false>(t, group, j, k));
      const uint4 w = drop_words(d, c >> 2, row);
      v[k] = word_of(w, c & 3) >= d.threshold ? v[k] * d.scale : 0.f;
    }
  }
}

// Sum (or largest) over the `group` threads of a row: shuffles, and for a
// group of several warps (then it is the block) one barrier; `slot` of shared
// memory is another one at each call that the last may still be read from.
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
  const int warps = group >> 5, lane = threadIdx.x & 31;
  v = lane < warps ? slot[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

// r = (ss / dim + eps)^(-1/2) of the row in v.  Where the squares leave the
// range of fp32 the sum is taken again of values scaled down by 2^-70 (exact),
// which the result is scaled by as well.
template <int VPT>
__device__ __forceinline__ float rstd_of(const float (&v)[VPT][8], int dim, float eps, int group,
                                         float *slots) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(v[j][k], v[j][k], ss);
  ss = over_group<false>(ss, group, slots);
  const float n = static_cast<float>(dim);
  // the same in every thread of a block-wide group; the smaller groups of a
  // warp shuffle together
  const bool far = !(ss <= 1e38f);
  if (!(group > 32 ? far : __any_sync(0xffffffffu, far))) return 1.f / sqrtf(ss / n + eps);
  float s2 = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float u = v[j][k] * 0x1p-70f;
      s2 = fmaf(u, u, s2);
    }
  s2 = over_group<false>(s2, group, slots + 32);
  return far ? 0x1p-70f / sqrtf(s2 / n + eps * 0x1p-140f) : 1.f / sqrtf(ss / n + eps);
}

// Forward: one row a group of threads.
template <class T, int VPT, bool AL, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_fwd(FwdArgs a) {
  __shared__ float slots[96];
  griddep_wait();
  griddep_launch_dependents();
  const int group = a.group;
  const int t = threadIdx.x % group;
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / group) + threadIdx.x / group;
  const bool live = row < a.rows;
  const int dim = live ? a.dim : 0;  // a group without a row holds zeros
  const Where at = where(live ? row : 0, a.inner);
  float v[VPT][8];
  {
    const T *x = static_cast<const T *>(a.x) + at.at(a.sx);
    Held<AL, T> hx[VPT], hr[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) fetch(hx[j], x, t, group, j, dim);
    if (a.res != nullptr) {
      const T *r = static_cast<const T *>(a.res) + at.at(a.sr);
#pragma unroll
      for (int j = 0; j < VPT; ++j) fetch(hr[j], r, t, group, j, dim);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) open(hx[j], t, group, j, dim, v[j]);
    if (a.dropped) {
      drop_resolve(a.drop);
#pragma unroll
      for (int j = 0; j < VPT; ++j) drop_vector<AL>(a.drop, row, t, group, j, v[j]);
    }
    if (a.res != nullptr) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float r[8];
        open(hr[j], t, group, j, dim, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += r[k];
      }
    }
    if (a.res != nullptr || a.dropped) {
      // the norm is of what the stream holds: rounded once, to the dtype
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = to_f32(from_f32<T>(v[j][k]));
      if (a.h != nullptr) {
        T *h = static_cast<T *>(a.h) + at.at(a.sh);
#pragma unroll
        for (int j = 0; j < VPT; ++j) put<AL>(h, t, group, j, dim, v[j]);
      }
    }
  }
  const float rstd = rstd_of(v, a.dim, a.eps, group, slots);
  if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float w[8];
    weight<AL, T>(a.w, a.w32, t, group, j, dim, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[j][k] = v[j][k] * rstd * w[k];
      top = fmaxf(top, fabsf(v[j][k]));
    }
  }
  if (a.y != nullptr) {
    T *y = static_cast<T *>(a.y) + at.at(a.sy);
#pragma unroll
    for (int j = 0; j < VPT; ++j) put<AL>(y, t, group, j, dim, v[j]);
  }
  if (a.codes == nullptr) return;
  top = over_group<true>(top, group, slots + 64);
  // an infinite row's scale is that of the largest finite number
  const int e = top <= 3.4028234e38f ? max(pow2_exponent(top), -126) : 120;
  const float inv = ldexpf(1.f, -e);
  if (live && t == 0) a.scale[row] = ldexpf(1.f, e);
  uint8_t *q = a.codes + row * a.dim;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if constexpr (AL) {
      const int c = (t + j * group) * 8;
      if (c < dim) {
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          p[k] = to_e4m3x2(make_float2(v[j][2 * k] * inv, v[j][2 * k + 1] * inv));
        *reinterpret_cast<uint2 *>(q + c) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = element<false>(t, group, j, k);
        if (c < dim) q[c] = to_e4m3(v[j][k] * inv);
      }
    }
  }
}

// Backward: blocks stay and take rows; each thread adds up dy h r of its
// columns over the rows that it took.
template <class T, int VPT, bool AL, int MAX>
__global__ void __launch_bounds__(MAX) k_norm_bwd(BwdArgs a) {
  __shared__ float slots[64];
  __shared__ float cols[kSmallBlock * VPT * 8];  // dw of the groups of a small block
  griddep_wait();
  griddep_launch_dependents();
  if (a.dropped) drop_resolve(a.drop);
  const int group = a.group;
  const int t = threadIdx.x % group, sub = threadIdx.x / group, subs = blockDim.x / group;
  float acc[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[j][k] = 0.f;
  int parity = 0;
  for (int64_t first = int64_t(blockIdx.x) * subs; first < a.rows; first += int64_t(gridDim.x) * subs) {
    const int64_t row = first + sub;
    const bool live = row < a.rows;
    const int dim = live ? a.dim : 0;
    const Where at = where(live ? row : 0, a.inner);
    Held<AL, T> hy[VPT], hh[VPT], hd[VPT];
    const T *dy = static_cast<const T *>(a.dy) + at.at(a.sdy);
    const T *h = static_cast<const T *>(a.h) + at.at(a.sh);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      fetch(hy[j], dy, t, group, j, dim);
      fetch(hh[j], h, t, group, j, dim);
    }
    if (a.dh != nullptr) {
      const T *dh = static_cast<const T *>(a.dh) + at.at(a.sdh);
#pragma unroll
      for (int j = 0; j < VPT; ++j) fetch(hd[j], dh, t, group, j, dim);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float g[VPT][8];
    float along = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float w[8], hat[8];
      weight<AL, T>(a.w, a.w32, t, group, j, dim, w);
      open(hy[j], t, group, j, dim, g[j]);
      open(hh[j], t, group, j, dim, hat);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        hat[k] *= rstd;
        acc[j][k] = fmaf(g[j][k], hat[k], acc[j][k]);
        g[j][k] *= w[k];
        along = fmaf(g[j][k], hat[k], along);
      }
    }
    along = over_group<false>(along, group, slots + 32 * parity) / static_cast<float>(a.dim);
    parity ^= 1;
    T *dx = static_cast<T *>(a.dx) + at.at(a.sdx);
    T *dres = a.dres != nullptr ? static_cast<T *>(a.dres) + at.at(a.sdr) : nullptr;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float d[8], hat[8];
      open(hh[j], t, group, j, dim, hat);
      if (a.dh != nullptr) {
        open(hd[j], t, group, j, dim, d);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = fmaf(rstd, g[j][k] - hat[k] * rstd * along, d[k]);
      if (dres != nullptr) put<AL>(dres, t, group, j, dim, d);
      if (a.dropped) drop_vector<AL>(a.drop, row, t, group, j, d);
      put<AL>(dx, t, group, j, dim, d);
    }
  }
  if (a.partial == nullptr) return;
  float *out = a.partial + int64_t(blockIdx.x) * a.dim;
  if (subs == 1) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) put<AL>(out, t, group, j, a.dim, acc[j]);
    return;
  }
  // several rows at a time: the groups' sums, added in their order
  const int width = group * VPT * 8;  // >= dim
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) cols[sub * width + element<AL>(t, group, j, k)] = acc[j][k];
  __syncthreads();
  for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
    float s = 0.f;
    for (int i = 0; i < subs; ++i) s += cols[i * width + c];
    out[c] = s;
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

// Threads of a row and vectors a thread.  `spread`: few rows, so as many
// threads as there are vectors.
struct Split {
  int group, vpt, block, per_block;  // per_block: rows
};
Split split_of(int dim, bool spread) {
  Split s;
  const int vectors = (dim + 7) / 8;
  s.vpt = spread && vectors <= 1024 ? 1 : vectors >= 4 * 16 ? 4 : vectors >= 2 * 16 ? 2 : 1;
  if (vectors > 2 * 1024 && s.vpt < 4) s.vpt = 4;
  const int threads = (vectors + s.vpt - 1) / s.vpt;
  if (threads <= 32) {
    s.group = 1;
    while (s.group < threads) s.group *= 2;
    s.block = kSmallBlock;
  } else {
    s.group = s.block = (threads + 31) / 32 * 32;
  }
  s.per_block = s.block / s.group;
  return s;
}

// Rows few enough to leave SMs without one: 2 a SM of the 152.
bool few_rows(int64_t rows) { return rows <= 304; }

// Blocks of the backward, each with a line of partial sums: four an SM where
// the rows go round (their registers fit five of 128 threads), and no more
// than there are rows.
constexpr int kBwdBlocks = 152 * 4;
int bwd_blocks(const Split &s, int64_t rows) {
  const int64_t n = (rows + s.per_block - 1) / s.per_block;
  return static_cast<int>(n < kBwdBlocks ? n : kBwdBlocks);
}

template <class T, bool AL>
cudaError_t launch_fwd(const FwdArgs &a, const Split &s, cudaStream_t st) {
  // (a block of over 256 threads has 64 registers a thread: dim over 8192 only)
  auto k = s.vpt == 1   ? k_norm_fwd<T, 1, AL, 1024>
           : s.vpt == 2 ? k_norm_fwd<T, 2, AL, 128>
           : s.block <= 256 ? k_norm_fwd<T, 4, AL, 256> : k_norm_fwd<T, 4, AL, 1024>;
  const int64_t blocks = (a.rows + s.per_block - 1) / s.per_block;
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(s.block), 0, st, a);
}
template <class T, bool AL>
cudaError_t launch_bwd(const BwdArgs &a, const Split &s, cudaStream_t st) {
  auto k = s.vpt == 1   ? k_norm_bwd<T, 1, AL, 1024>
           : s.vpt == 2 ? k_norm_bwd<T, 2, AL, 128>
           : s.block <= 256 ? k_norm_bwd<T, 4, AL, 256> : k_norm_bwd<T, 4, AL, 1024>;
  return launch_pdl(k, dim3(bwd_blocks(s, a.rows)), dim3(s.block), 0, st, a);
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
  lora_status_t add(const void *p, const int64_t *s, const char *name, bool out, Rows &rows) {
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
  LORA_TRY(ts.add(x, sh->x, "x", false, a.sx));
  if (residual != nullptr) LORA_TRY(ts.add(residual, sh->residual, "residual", false, a.sr));
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
  const Split s = split_of(sh->dim, few_rows(rows));
  a.group = s.group;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_NORM, st, "norm", [&] {
    if (dtype == LORA_BF16)
      return ts.vec ? launch_fwd<__nv_bfloat16, true>(a, s, st) : launch_fwd<__nv_bfloat16, false>(a, s, st);
    return ts.vec ? launch_fwd<float, true>(a, s, st) : launch_fwd<float, false>(a, s, st);
  });
}

size_t lora_norm_workspace_bytes(const lora_norm_t *sh, int with_dw) {
  clear_error();
  if (check_shape(sh, LORA_BF16) != LORA_OK || !with_dw) return 0;
  const int64_t rows = sh->outer * sh->inner;
  return size_t(bwd_blocks(split_of(sh->dim, few_rows(rows)), rows)) * sh->dim * sizeof(float);
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
  const Split s = split_of(sh->dim, few_rows(rows));
  const int blocks = bwd_blocks(s, rows);
  bool vec = sh->dim % 8 == 0;
  if (rows > 0) {
    Tensors ts = {sh, dtype == LORA_BF16 ? 2 : 4, vec};
    LORA_TRY(ts.add(dy, sh->dy, "dy", false, a.sdy));
    LORA_TRY(ts.add(h, sh->h, "h", false, a.sh));
    if (dh != nullptr) LORA_TRY(ts.add(dh, sh->dh, "dh", false, a.sdh));
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
    LORA_TRY(run(LORA_K_NORM_BWD, st, "norm backward", [&] {
      if (dtype == LORA_BF16)
        return vec ? launch_bwd<__nv_bfloat16, true>(a, s, st) : launch_bwd<__nv_bfloat16, false>(a, s, st);
      return vec ? launch_bwd<float, true>(a, s, st) : launch_bwd<float, false>(a, s, st);
    }));
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
