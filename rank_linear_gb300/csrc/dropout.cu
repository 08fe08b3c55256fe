// dropout.cu -- dropout from a counter-based generator (include/lora_dropout.h;
// the Unsloth essay's recipe table names the rate).
//
// y = keep ? x * scale : 0 with the mask made from (seed, offset, row, column)
// by both directions.  An element moves 4 bytes (bf16) or 8, and costs 1/4 of a
// Philox call, some 17 instructions: the rates of memory and of the integer
// products lie close together.
#include <cmath>

#include "dropout.cuh"
#include "host.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void *x;
  void *y;
  int64_t rows, xs, ys, total;  // total: work items
  uint32_t cols, per_row;       // items a row
  uint32_t mul;                 // item / per_row = item * mul >> shift for
  int shift;                    // items below 2^31
  DropArgs drop;
};

// Item -> (row, item within the row).  The quotient of a 31-bit number by a
// constant is a product and a shift (Granlund and Montgomery, 1994).
__device__ __forceinline__ void place(const Args &a, int64_t item, int64_t &row, uint32_t &i) {
  if (a.total < (int64_t(1) << 31)) {
    const uint32_t r = static_cast<uint32_t>(uint64_t(item) * a.mul >> a.shift);
    row = r;
    i = static_cast<uint32_t>(item) - r * a.per_row;
  } else {
    row = item / a.per_row;
    i = static_cast<uint32_t>(item - row * a.per_row);
  }
}

// Rows of whole, aligned vectors of eight: each thread has kItems of them in
// flight before it makes their masks.
template <class T, int kItems>
__global__ void __launch_bounds__(kThreads) k_dropout(const __grid_constant__ Args a) {
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  Raw8<T> in[kItems];
  int64_t row[kItems];
  uint32_t v[kItems];
  const int64_t first = int64_t(blockIdx.x) * (kThreads * kItems) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int64_t item = first + j * kThreads;
    if (item < a.total) {
      place(a, item, row[j], v[j]);
      in[j].load(static_cast<const T *>(a.x) + row[j] * a.xs + int64_t(v[j]) * 8);
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (first + j * kThreads >= a.total) break;
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = in[j].pair(i);
    drop8(a.drop, now, v[j], row[j], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) in[j].set(i, f[i]);
    in[j].store(static_cast<T *>(a.y) + row[j] * a.ys + int64_t(v[j]) * 8);
  }
}

// Any width and alignment: four columns (one Philox call) a thread.
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const __grid_constant__ Args a) {
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  const int64_t item = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= a.total) return;
  int64_t row;
  uint32_t b;
  place(a, item, row, b);
  const T *x = static_cast<const T *>(a.x) + row * a.xs + int64_t(b) * 4;
  T *y = static_cast<T *>(a.y) + row * a.ys + int64_t(b) * 4;
  const uint32_t n = a.cols - b * 4;  // 4 columns, fewer at the row's end
  float f[4];
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) f[i] = i < n ? to_f32(x[i]) : 0.f;
  const uint4 w = drop_words(a.drop, now, b, row);
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    if (i < n) y[i] = from_f32<T>(drop1(a.drop, word_of(w, i), f[i]));
}

template <class T>
cudaError_t launch_dropout(Args a, bool vec, cudaStream_t s) {
  a.per_row = vec ? a.cols / 8 : (a.cols + 3) / 4;
  a.total = a.rows * a.per_row;
  int l = 0;
  while ((uint64_t(1) << l) < a.per_row) ++l;
  a.shift = 31 + l;
  a.mul = static_cast<uint32_t>((uint64_t(1) << a.shift) / a.per_row + 1);
  const int64_t per_block = vec ? kThreads * 2 : kThreads;
  const int64_t blocks = (a.total + per_block - 1) / per_block;
  const dim3 grid(static_cast<unsigned>(blocks));
  return vec ? launch_pdl(k_dropout<T, 2>, grid, dim3(kThreads), 0, s, a)
             : launch_pdl(k_dropout_any<T>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

lora_status_t drop_args(const lora_dropout_t *d, DropArgs &out) {
  out = DropArgs{};
  if (d == nullptr) return LORA_OK;
  if (!(d->p >= 0.0) || !(std::nearbyint(d->p * 0x1p32) < 0x1p32))
    return fail(LORA_ERR_INVALID_ARG, "dropout p = %g is not in [0, 1)", d->p);
  if (reinterpret_cast<uintptr_t>(d->state) % 8 != 0)
    return fail(LORA_ERR_INVALID_ARG, "the dropout's state is not 8-byte aligned");
  out.threshold = static_cast<uint32_t>(std::nearbyint(d->p * 0x1p32));
  out.scale = static_cast<float>(0x1p32 / (0x1p32 - out.threshold));
  out.seed = d->seed;
  out.offset = d->offset;
  out.state = d->state;
  drop_keys(out);
  return LORA_OK;
}

}  // namespace lora

using namespace lora;

extern "C" lora_status_t lora_dropout(const void *x, int64_t rows, int64_t cols, int64_t x_stride,
                                      int64_t y_stride, const lora_dropout_t *dropout,
                                      lora_dtype_t dtype, void *y, void *stream) {
  clear_error();
  if (dropout == nullptr) return fail(LORA_ERR_INVALID_ARG, "dropout is NULL");
  if (dtype != LORA_BF16 && dtype != LORA_FP32)
    return fail(LORA_ERR_INVALID_ARG, "dtype %d is not LORA_BF16 or LORA_FP32", int(dtype));
  if (rows < 0 || cols < 0) return fail(LORA_ERR_INVALID_ARG, "rows or cols is negative");
  if (cols >= (int64_t(1) << 31) || rows > (int64_t(1) << 36) ||
      (cols > 0 && rows > (int64_t(1) << 40) / cols))
    return fail(LORA_ERR_UNSUPPORTED,
                "rows of 2^31 elements or more, over 2^36 rows, or over 2^40 elements");
  Args a = {};
  LORA_TRY(drop_args(dropout, a.drop));
  if (rows == 0 || cols == 0) return LORA_OK;
  if (x == nullptr || y == nullptr) return fail(LORA_ERR_INVALID_ARG, "x or y is NULL");
  const int es = dtype == LORA_BF16 ? 2 : 4;
  auto aligned = [](const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!aligned(x, es) || !aligned(y, es))
    return fail(LORA_ERR_INVALID_ARG, "x or y is not aligned to its type");
  if (rows > 1 && y_stride < cols)
    return fail(LORA_ERR_INVALID_ARG, "the rows of y overlap (stride %lld)", (long long)y_stride);
  if (x == y && rows > 1 && x_stride != y_stride)
    return fail(LORA_ERR_INVALID_ARG, "y is x with another stride");
  a.x = x;
  a.y = y;
  a.rows = rows;
  a.cols = static_cast<uint32_t>(cols);
  a.xs = rows > 1 ? x_stride : 0;
  a.ys = rows > 1 ? y_stride : 0;
  const int per16 = 16 / es;
  const bool vec = cols % 8 == 0 && aligned(x, 16) && aligned(y, 16) && a.xs % per16 == 0 &&
                   a.ys % per16 == 0;
  DevInfo di;
  LORA_TRY(device_info(di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run(LORA_K_DROPOUT, st, "dropout", [&] {
    return dtype == LORA_BF16 ? launch_dropout<__nv_bfloat16>(a, vec, st)
                              : launch_dropout<float>(a, vec, st);
  });
}
