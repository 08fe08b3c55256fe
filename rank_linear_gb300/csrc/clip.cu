// clip.cu -- global gradient norm and clipping (include/lora_clip.h).
//
// Two passes, both bound by memory: one reads every gradient and leaves the
// norm and the factor in the plan, the other scales.  The plan cuts the
// tensors into chunks of 16 KB (4 KB where that would leave SMs without
// work), one 32-byte record each, so that a block finds its work with one
// load whatever the number of tensors; the record of a block's next chunk is
// loaded before the present one is read.  The scaling pass visits the chunks
// in reverse order: those read last are still in L2.
//
// Measured, both passes: 84 MB of bf16 in 448 tensors 42 us (read twice and
// written once, 6.0 TB/s), 2.3 GB 1040 us (6.7 TB/s, a copy's bandwidth),
// 2.6 MB in 14 tensors 10 us (two launches).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "host.h"
#include "lora_clip.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256, kVecs = 4;  // 16-byte vectors of a thread per 16 KB chunk
constexpr int kNormBlocks = 4, kClipBlocks = 6, kMaxBlocks = 1024;  // blocks of an SM (two), of all

struct Chunk {
  const void *in;
  void *out;
  int count, dtype;
  int64_t pad;
};
static_assert(sizeof(Chunk) == 32, "chunk record");

// A block's part of the norm: in fp32 (a pair for the sum of squares), and in
// fp64, which counts where the fp32 one is out of range (see out_of_range).
struct Partial {
  float hi, lo;
  double full;
};
struct PlanHead {
  unsigned ticket;  // blocks of the norm pass done; 0 between calls
  int pad[3];
  Partial partial[kMaxBlocks];
};
static_assert(sizeof(PlanHead) % 16 == 0, "chunks stay aligned");

__device__ __forceinline__ Chunk load_chunk(const Chunk *p) {
  Chunk c;
  const int4 a = __ldcg(reinterpret_cast<const int4 *>(p));
  const int4 b = __ldcg(reinterpret_cast<const int4 *>(p) + 1);
  reinterpret_cast<int4 *>(&c)[0] = a;
  reinterpret_cast<int4 *>(&c)[1] = b;
  return c;
}

// Elements before the first 16-byte boundary (at most n), and vectors after.
template <int ES>
__device__ __forceinline__ void split_run(const void *p, int n, int &head, int &vecs) {
  head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / ES);
  vecs = (n - head) / (16 / ES);
}

__device__ __forceinline__ float2 bf2(unsigned u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// The elements of one 16-byte vector as floats.
template <bool BF>
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[BF ? 8 : 4]) {
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) {
      const float2 t = bf2(w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}

// fp32 sums of squares outside these bounds may have lost squares to
// underflow or overflow (each square kept to 2^-24 above 2^-126).
constexpr float kSafeLow = 1e-30f, kSafeHigh = 1e30f;

// A thread's sum: fast as an unevaluated sum of two fp32 (fp64 adds are some
// 30 times dearer here), wide for what does not fit fp32.
struct Sum {
  float hi = 0.f, lo = 0.f;
  double wide = 0.0;
};
// hi + lo += x + y (|x| arbitrary): the exact sum of hi and x, its error kept.
__device__ __forceinline__ void add_to(float &hi, float &lo, float x, float y) {
  const float s = hi + x, t = s - hi;
  lo += ((hi - (s - t)) + (x - t)) + y;
  hi = s;
}

// A chunk's vectors (of its input).
struct Held {
  uint4 v[kVecs];
};
template <int ES>
__device__ __forceinline__ const uint4 *body_of(const Chunk &c, int &head, int &vecs) {
  split_run<ES>(c.in, c.count, head, vecs);
  return reinterpret_cast<const uint4 *>(static_cast<const char *>(c.in) + head * ES);
}
__device__ __forceinline__ void hold(const Chunk &c, Held &h) {
  int head, vecs;
  const uint4 *body = c.dtype == LORA_BF16 ? body_of<2>(c, head, vecs) : body_of<4>(c, head, vecs);
  body += threadIdx.x;
  if (vecs == kVecs * kThreads) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) h.v[u] = __ldcg(body + u * kThreads);
  } else {
    vecs -= threadIdx.x;
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      h.v[u] = u * kThreads < vecs ? __ldcg(body + u * kThreads) : make_uint4(0, 0, 0, 0);
  }
}

template <bool BF, bool LARGEST>
__device__ __forceinline__ void add_chunk(const Chunk &c, const Held &h, Sum &acc) {
  constexpr int N = BF ? 8 : 4, ES = 16 / N;
  int head, vecs;
  split_run<ES>(c.in, c.count, head, vecs);
  // the elements outside whole vectors: fewer than 2 N of them
  const int tid = threadIdx.x, rest = c.count - vecs * N;
  float lone = 0.f;
  if (tid < rest) {
    const int i = tid < head ? tid : tid + vecs * N;
    if constexpr (BF)
      lone = __bfloat162float(static_cast<const __nv_bfloat16 *>(c.in)[i]);
    else
      lone = static_cast<const float *>(c.in)[i];
  }
  if constexpr (LARGEST) {
    float m = acc.hi;
    auto top = [&](float x) {  // fmaxf would drop NaN
      x = fabsf(x);
      if (!(x <= m)) m = (m != m) ? m : x;
    };
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float f[N];
      unpack<BF>(h.v[u], f);
#pragma unroll
      for (int e = 0; e < N; ++e) top(f[e]);
    }
    top(lone);
    acc.hi = m;
  } else {
    float s0 = lone * lone, s1 = 0.f;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float f[N];
      unpack<BF>(h.v[u], f);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        s0 = fmaf(f[e], f[e], s0);
        s1 = fmaf(f[e + 1], f[e + 1], s1);
      }
    }
    const float s = s0 + s1;
    if (s >= kSafeLow && s <= kSafeHigh) {
      add_to(acc.hi, acc.lo, s, 0.f);
    } else {  // all zero, far off scale, or not finite: again in fp64
      unsigned any = __float_as_uint(lone) << 1;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) any |= h.v[u].x | h.v[u].y | h.v[u].z | h.v[u].w;
      if (any != 0) {
        double d = static_cast<double>(lone) * lone;
        const uint4 *body = body_of<ES>(c, head, vecs);
#pragma unroll 1
        for (int i = tid; i < vecs; i += kThreads) {
          float f[N];
          unpack<BF>(__ldcg(body + i), f);
#pragma unroll
          for (int e = 0; e < N; ++e) d += static_cast<double>(f[e]) * f[e];
        }
        acc.wide += d;
      }
    }
  }
}

// NaN wins.
__device__ __forceinline__ float larger(float a, float b) {
  return (a != a) ? a : (b <= a ? a : b);
}

// The threads' values in every thread; the order depends on the block size only.
template <bool LARGEST>
__device__ float2 join_block(float hi, float lo) {
  __shared__ float2 part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(~0u, hi, o);
    if constexpr (LARGEST)
      hi = larger(hi, x);
    else
      add_to(hi, lo, x, __shfl_xor_sync(~0u, lo, o));
  }
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(hi, lo);
  __syncthreads();
  float2 v = part[0];
  for (int i = 1; i < kThreads / 32; ++i) {
    if constexpr (LARGEST)
      v.x = larger(v.x, part[i].x);
    else
      add_to(v.x, v.y, part[i].x, part[i].y);
  }
  __syncthreads();
  return v;
}
__device__ double join_block(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kThreads / 32; ++i) v += part[i];
  __syncthreads();
  return v;
}

// Joins the blocks' parts in the order of their numbers; the norm, in every
// thread.
template <bool LARGEST>
__device__ float join_parts(const PlanHead *head, int blocks) {
  float hi = 0.f, lo = 0.f;
  for (int b = threadIdx.x; b < blocks; b += kThreads) {
    const float2 v = __ldcg(reinterpret_cast<const float2 *>(&head->partial[b]));
    if constexpr (LARGEST)
      hi = larger(hi, v.x);
    else
      add_to(hi, lo, v.x, v.y);
  }
  const float2 v = join_block<LARGEST>(hi, lo);
  if constexpr (LARGEST) return v.x;
  const float total = v.x + v.y;
  if (total > kSafeLow && total < kSafeHigh) return sqrtf(total);
  // nothing at all, far off scale, or not finite
  double full = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kThreads) full += __ldcg(&head->partial[b].full);
  return static_cast<float>(sqrt(join_block(full)));
}

// JOIN: the last block done also joins the parts into norm[0] (else the
// clipping pass does, in each of its blocks: cheaper than the ticket and one
// block's work behind it).
template <bool LARGEST, bool JOIN>
__global__ void __launch_bounds__(kThreads, kNormBlocks) k_grad_norm(PlanHead *head, const Chunk *chunks,
                                                        int n, float *norm) {
  __shared__ bool last;
  griddep_wait();
  griddep_launch_dependents();
  Sum sum;
  const int step = gridDim.x;
  int i = blockIdx.x;
  if (i < n) {
    // a chunk's vectors are asked for before the one ahead of it is summed,
    // its record before that
    Chunk c = load_chunk(chunks + i), cn = c;
    if (i + step < n) cn = load_chunk(chunks + i + step);
    Held h, hn;
    hold(c, h);
    while (true) {
      Chunk c2 = cn;
      if (i + 2 * step < n) c2 = load_chunk(chunks + i + 2 * step);
      if (i + step < n) hold(cn, hn);
      if (c.dtype == LORA_BF16)
        add_chunk<true, LARGEST>(c, h, sum);
      else
        add_chunk<false, LARGEST>(c, h, sum);
      i += step;
      if (i >= n) break;
      c = cn;
      cn = c2;
      h = hn;
    }
  }
  float2 v = join_block<LARGEST>(sum.hi, sum.lo);
  Partial p = {v.x, v.y, 0.0};
  if constexpr (!LARGEST) {
    const bool wide = __syncthreads_or(sum.wide != 0.0);  // NaN is not 0
    double full = 0.0;
    if (wide) full = join_block(sum.wide);
    p.full = static_cast<double>(v.x) + v.y + full;
    if (wide) {  // as fp32 has it: out of its safe range, or good to 2^-24
      p.hi = static_cast<float>(p.full);
      p.lo = p.hi - p.hi != 0.f ? 0.f : static_cast<float>(p.full - p.hi);
    }
  }
  if (threadIdx.x == 0) head->partial[blockIdx.x] = p;
  if constexpr (JOIN) {
    if (threadIdx.x == 0) {
      __threadfence();
      last = atomicAdd(&head->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    const float total = join_parts<LARGEST>(head, gridDim.x);
    if (threadIdx.x == 0) {
      norm[0] = total;
      head->ticket = 0;
    }
  }
}

__device__ __forceinline__ bool aligned_alike(const Chunk &c) {
  return ((reinterpret_cast<uintptr_t>(c.in) ^ reinterpret_cast<uintptr_t>(c.out)) & 15) == 0;
}

template <bool BF>
__device__ __forceinline__ void scale_chunk(const Chunk &c, const Held &h, float f) {
  constexpr int N = BF ? 8 : 4, ES = 16 / N;
  using T = typename std::conditional<BF, __nv_bfloat16, float>::type;
  const T *in = static_cast<const T *>(c.in);
  T *out = static_cast<T *>(c.out);
  auto one = [&](int i) {
    if constexpr (BF)
      out[i] = __float2bfloat16_rn(__bfloat162float(in[i]) * f);
    else
      out[i] = in[i] * f;
  };
  const int tid = threadIdx.x;
  if (!aligned_alike(c)) {
#pragma unroll 4
    for (int i = tid; i < c.count; i += kThreads) one(i);
    return;
  }
  int head, vecs;
  split_run<ES>(c.in, c.count, head, vecs);
  uint4 *dst = reinterpret_cast<uint4 *>(out + head);
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int i = tid + u * kThreads;
    if (i >= vecs) continue;
    float x[N];
    unpack<BF>(h.v[u], x);
    uint4 o;
    unsigned *w = reinterpret_cast<unsigned *>(&o);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e] * f, x[2 * e + 1] * f);
        w[e] = *reinterpret_cast<const unsigned *>(&p);
      } else {
        w[e] = __float_as_uint(x[e] * f);
      }
    }
    __stcs(dst + i, o);  // read by no one here: leaves L2 to the gradients
  }
  if (tid < c.count - vecs * N) one(tid < head ? tid : tid + vecs * N);
}

template <bool LARGEST>
__global__ void __launch_bounds__(kThreads, kClipBlocks) k_grad_clip(const PlanHead *head,
                                                           const Chunk *chunks, int n, int parts,
                                                           float max_norm, float *norm) {
  // Records and gradients do not depend on the norm pass (which let this
  // kernel start when all before it was done): the first chunk is asked for
  // ahead of the wait.
  int i = n - 1 - static_cast<int>(blockIdx.x);
  Chunk c = {};
  Held h;
  if (i >= 0) {
    c = load_chunk(chunks + i);
    hold(c, h);
  }
  griddep_wait();
  griddep_launch_dependents();
  const float total = join_parts<LARGEST>(head, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = total;
  const float by = max_norm / (total + 1e-6f);
  const float f = by > 1.f ? 1.f : by;  // NaN stays NaN
  while (i >= 0) {
    const int next = i - static_cast<int>(gridDim.x);
    Chunk cn = {};
    if (next >= 0) cn = load_chunk(chunks + next);
    if (f != 1.f || c.in != c.out) {
      if (c.dtype == LORA_BF16)
        scale_chunk<true>(c, h, f);
      else
        scale_chunk<false>(c, h, f);
    }
    c = cn;
    if (next >= 0 && (f != 1.f || c.in != c.out)) hold(c, h);
    i = next;
  }
}

// ---------------------------------------------------------------- host
lora_status_t check_tensors(const lora_clip_tensor_t *t, int n, int64_t *bytes) {
  if (n < 0 || n > (1 << 24)) return fail(LORA_ERR_INVALID_ARG, "n = %d tensors", n);
  if (n > 0 && t == nullptr) return fail(LORA_ERR_INVALID_ARG, "tensors is NULL");
  *bytes = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].dtype != LORA_BF16 && t[i].dtype != LORA_FP32)
      return fail(LORA_ERR_INVALID_ARG, "tensor %d: dtype %d is not LORA_BF16 or LORA_FP32", i,
                  int(t[i].dtype));
    const int es = t[i].dtype == LORA_BF16 ? 2 : 4;
    if (t[i].count < 0 || t[i].count > (int64_t(1) << 40))
      return fail(LORA_ERR_INVALID_ARG, "tensor %d: %lld elements", i, (long long)t[i].count);
    if (t[i].count == 0) continue;
    if (t[i].in == nullptr || t[i].out == nullptr)
      return fail(LORA_ERR_INVALID_ARG, "tensor %d: NULL", i);
    if (reinterpret_cast<uintptr_t>(t[i].in) % es || reinterpret_cast<uintptr_t>(t[i].out) % es)
      return fail(LORA_ERR_INVALID_ARG, "tensor %d is not aligned to its type", i);
    *bytes += t[i].count * es;
  }
  if (*bytes > (int64_t(1) << 42))
    return fail(LORA_ERR_UNSUPPORTED, "more than 2^42 bytes of gradients");
  return LORA_OK;
}

// No output may share memory with another tensor (but for its own input, in
// place): blocks read and write them in any order.  One sweep over the tensors
// by address.
lora_status_t check_overlap(const lora_clip_tensor_t *t, int n) {
  struct Run {
    uintptr_t from, to;
    int tensor;
    bool written;
  };
  try {
    std::vector<Run> runs;
    runs.reserve(2 * size_t(n));
    for (int i = 0; i < n; ++i) {
      const uintptr_t size = uintptr_t(t[i].count) * (t[i].dtype == LORA_BF16 ? 2 : 4);
      if (size == 0) continue;
      const uintptr_t in = reinterpret_cast<uintptr_t>(t[i].in);
      const uintptr_t out = reinterpret_cast<uintptr_t>(t[i].out);
      runs.push_back({out, out + size, i, true});
      if (in != out) runs.push_back({in, in + size, i, false});
    }
    std::sort(runs.begin(), runs.end(), [](const Run &a, const Run &b) { return a.from < b.from; });
    Run any = {0, 0, -1, false}, written = any;  // of those before, the one that ends last
    for (const Run &r : runs) {
      const Run &other = r.written ? any : written;
      if (r.from < other.to)
        return fail(LORA_ERR_INVALID_ARG, "the output of tensor %d shares memory with tensor %d",
                    r.written ? r.tensor : other.tensor, r.written ? other.tensor : r.tensor);
      if (r.to > any.to) any = r;
      if (r.written && r.to > written.to) written = r;
    }
  } catch (const std::bad_alloc &) {
    return fail(LORA_ERR_WORKSPACE, "no host memory to compare %d tensors", n);
  }
  return LORA_OK;
}

// 4 KB chunks (one vector a thread) where 16 KB ones would not give a GB300's
// 152 SMs four blocks each.
int chunk_bytes(int64_t total) { return total < int64_t(152) * 4 * 16384 ? 4096 : 16384; }

int64_t count_chunks(const lora_clip_tensor_t *t, int n, int cb) {
  int64_t c = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t per = cb / (t[i].dtype == LORA_BF16 ? 2 : 4);
    c += (t[i].count + per - 1) / per;
  }
  return c;
}

lora_status_t check_plan(const void *plan, size_t bytes, int largest, const float *norm, int *n) {
  if (plan == nullptr || norm == nullptr)
    return fail(LORA_ERR_INVALID_ARG, "plan or norm is NULL");
  if (reinterpret_cast<uintptr_t>(plan) % 16 || reinterpret_cast<uintptr_t>(norm) % 4)
    return fail(LORA_ERR_INVALID_ARG, "plan (16 bytes) or norm (4 bytes) is not aligned");
  if ((largest | 1) != 1) return fail(LORA_ERR_INVALID_ARG, "largest = %d is not 0 or 1", largest);
  if (bytes < sizeof(PlanHead) || (bytes - sizeof(PlanHead)) % sizeof(Chunk) != 0 ||
      (bytes - sizeof(PlanHead)) / sizeof(Chunk) > size_t(INT32_MAX) / 2)
    return fail(LORA_ERR_INVALID_ARG, "%zu bytes is no plan's size", bytes);
  *n = static_cast<int>((bytes - sizeof(PlanHead)) / sizeof(Chunk));
  return LORA_OK;
}

int norm_blocks(const DevInfo &di, int n) {
  const int most = di.sms * kNormBlocks < kMaxBlocks ? di.sms * kNormBlocks : kMaxBlocks;
  return n < 1 ? 1 : n < most ? n : most;
}
lora_status_t norm_pass(const DevInfo &di, PlanHead *head, int n, int largest, bool join,
                        float *norm, cudaStream_t st) {
  const Chunk *chunks = reinterpret_cast<const Chunk *>(head + 1);
  auto *kernel = largest ? (join ? k_grad_norm<true, true> : k_grad_norm<true, false>)
                         : (join ? k_grad_norm<false, true> : k_grad_norm<false, false>);
  return run(LORA_K_GRAD_NORM, st, "gradient norm", [&] {
    return launch_pdl(kernel, dim3(norm_blocks(di, n)), dim3(kThreads), 0, st, head, chunks, n, norm);
  });
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_clip_plan_bytes(const lora_clip_tensor_t *tensors, int n) {
  clear_error();
  int64_t total = 0;
  if (check_tensors(tensors, n, &total) != LORA_OK) return 0;
  return sizeof(PlanHead) + size_t(count_chunks(tensors, n, chunk_bytes(total))) * sizeof(Chunk);
}

lora_status_t lora_clip_plan_build(const lora_clip_tensor_t *tensors, int n, void *image,
                                   size_t image_bytes) {
  clear_error();
  int64_t total = 0;
  LORA_TRY(check_tensors(tensors, n, &total));
  LORA_TRY(check_overlap(tensors, n));
  const int cb = chunk_bytes(total);
  const size_t need = sizeof(PlanHead) + size_t(count_chunks(tensors, n, cb)) * sizeof(Chunk);
  if (image == nullptr || image_bytes != need)
    return fail(LORA_ERR_WORKSPACE, "a plan image of %zu bytes is needed, got %zu%s", need,
                image_bytes, image == nullptr ? " (NULL)" : "");
  uint8_t *out = static_cast<uint8_t *>(image);
  std::memset(out, 0, sizeof(PlanHead));
  out += sizeof(PlanHead);
  for (int i = 0; i < n; ++i) {
    const int es = tensors[i].dtype == LORA_BF16 ? 2 : 4;
    const int64_t per = cb / es;
    for (int64_t at = 0; at < tensors[i].count; at += per) {
      const int64_t left = tensors[i].count - at;
      Chunk c = {};
      c.in = static_cast<const char *>(tensors[i].in) + at * es;
      c.out = static_cast<char *>(tensors[i].out) + at * es;
      c.count = static_cast<int>(left < per ? left : per);
      c.dtype = tensors[i].dtype;
      std::memcpy(out, &c, sizeof(c));
      out += sizeof(c);
    }
  }
  return LORA_OK;
}

lora_status_t lora_clip_norm(void *plan, size_t plan_bytes, int largest, float *norm,
                             void *stream) {
  clear_error();
  int n = 0;
  LORA_TRY(check_plan(plan, plan_bytes, largest, norm, &n));
  DevInfo di;
  LORA_TRY(device_info(di));
  return norm_pass(di, static_cast<PlanHead *>(plan), n, largest, true, norm,
                   static_cast<cudaStream_t>(stream));
}

lora_status_t lora_clip(void *plan, size_t plan_bytes, float max_norm, int largest, float *norm,
                        void *stream) {
  clear_error();
  int n = 0;
  LORA_TRY(check_plan(plan, plan_bytes, largest, norm, &n));
  if (!(max_norm >= 0.f)) return fail(LORA_ERR_INVALID_ARG, "max_norm must be >= 0");
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  PlanHead *head = static_cast<PlanHead *>(plan);
  if (n == 0) return norm_pass(di, head, n, largest, true, norm, st);
  LORA_TRY(norm_pass(di, head, n, largest, false, norm, st));
  const Chunk *chunks = reinterpret_cast<const Chunk *>(head + 1);
  const int blocks = n < di.sms * kClipBlocks ? n : di.sms * kClipBlocks;
  return run(LORA_K_GRAD_CLIP, st, "gradient clip", [&] {
    return launch_pdl(largest ? k_grad_clip<true> : k_grad_clip<false>, dim3(blocks),
                      dim3(kThreads), 0, st, head, chunks, n, norm_blocks(di, n), max_norm, norm);
  });
}

}  // extern "C"
