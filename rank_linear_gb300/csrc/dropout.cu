// dropout.cu -- dropout from a counter-based generator (include/lora_dropout.h;
// the Unsloth essay's recipe table names the rate).
//
// y = keep ? x * scale : 0 with the mask made from (seed, offset, row, column)
// by both directions.  An element moves 4 bytes (bf16) or 8, and takes a quarter
// of the generator's ten rounds: 1.73e12 words a second is all that an otherwise
// empty loop of them makes on the 152 SMs (the 32 x 32 -> 64 products bound it),
// and 1.70e12 elements of bf16 a second is what memory moves.  So what is not the
// generator is kept small: a block's rows and addresses are worked out once, and
// where the block has one row, the row's share of the first two rounds as well.
#include <cmath>

#include "dropout.cuh"
#include "host.h"
#include "ptx.cuh"

namespace lora {
namespace {

struct Args {
  const void *x;
  void *y;
  int64_t rows, xs, ys;
  uint32_t cols, units;  // units of a row: eight columns, or four (any alignment)
  // A block takes `segment` units of one row (chunks of them make a row), kItems a
  // thread, and kRows rows; or, where a row has few, 2^lanes threads a row and two rows each.
  uint32_t chunks, segment;
  int lanes;
  DropArgs drop;
};

// Unit u of a row.
template <class T, bool VEC>
struct Unit;
template <class T>
struct Unit<T, true> {
  Raw8<T> v;
  __device__ __forceinline__ void load(const T *row, uint32_t u, uint32_t) { v.load(row + u * 8); }
  __device__ __forceinline__ void drop(const Args &a, const DropNow &now, uint32_t u, int64_t row) {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v.pair(i);
    drop8(a.drop, now, u, row, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.set(i, f[i]);
  }
  __device__ __forceinline__ void store(T *row, uint32_t u, uint32_t) const { v.store(row + u * 8); }
};
template <class T>
struct Unit<T, false> {
  float f[4];
  __device__ __forceinline__ void load(const T *row, uint32_t u, uint32_t cols) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) f[i] = u * 4 + i < cols ? to_f32(row[u * 4 + i]) : 0.f;
  }
  __device__ __forceinline__ void drop(const Args &a, const DropNow &now, uint32_t u, int64_t row) {
    const uint4 w = drop_words(a.drop, now, u, row);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) f[i] = drop1(a.drop, word_of(w, i), f[i]);
  }
  __device__ __forceinline__ void store(T *row, uint32_t u, uint32_t cols) const {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (u * 4 + i < cols) row[u * 4 + i] = from_f32<T>(f[i]);
  }
};

constexpr int kItems = 2;  // units a thread and row (four: 5 % longer, fewer threads fit)
constexpr int kRows = 4;   // rows a block: their common costs are shared

// Rows of many units: the same segment of kRows rows a block, the next row's units
// on their way while the masks of one are made.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) k_dropout(const __grid_constant__ Args a) {
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  int64_t row = int64_t(blockIdx.x / a.chunks) * kRows;
  const uint32_t first = (blockIdx.x % a.chunks) * a.segment;
  const uint32_t end = min(first + a.segment, a.units);
  const int64_t last = row + kRows < a.rows ? row + kRows : a.rows;
  const T *x = static_cast<const T *>(a.x) + row * a.xs;
  T *y = static_cast<T *>(a.y) + row * a.ys;
  Unit<T, VEC> in[kItems], next[kItems];
  auto load = [&](Unit<T, VEC> (&v)[kItems], const T *from) {
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const uint32_t u = first + threadIdx.x + j * blockDim.x;
      if (u < end) v[j].load(from, u, a.cols);
    }
  };
  load(in, x);
#pragma unroll 1
  for (; row < last; ++row) {
    x += a.xs;
    if (row + 1 < last) load(next, x);
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const uint32_t u = first + threadIdx.x + j * blockDim.x;
      if (u >= end) break;
      in[j].drop(a, now, u, row);
      in[j].store(y, u, a.cols);
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) in[j] = next[j];
    y += a.ys;
  }
}

// Rows of few units: several a block.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) k_dropout_rows(const __grid_constant__ Args a) {
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  const uint32_t u = threadIdx.x & ((1u << a.lanes) - 1u), at_once = 256u >> a.lanes;
  const int64_t first = int64_t(blockIdx.x) * (2 * at_once) + (threadIdx.x >> a.lanes);
  if (u >= a.units) return;
  Unit<T, VEC> in[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t row = first + j * at_once;
    if (row < a.rows) in[j].load(static_cast<const T *>(a.x) + row * a.xs, u, a.cols);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t row = first + j * at_once;
    if (row >= a.rows) break;
    in[j].drop(a, now, u, row);
    in[j].store(static_cast<T *>(a.y) + row * a.ys, u, a.cols);
  }
}

template <class T, bool VEC>
cudaError_t launch_dropout(Args a, cudaStream_t s) {
  a.units = VEC ? a.cols / 8 : (a.cols + 3) / 4;
  if (a.units <= 128) {
    a.lanes = 0;
    while ((1u << a.lanes) < a.units) ++a.lanes;
    const int64_t per = 2 * (256 >> a.lanes);
    return launch_pdl(k_dropout_rows<T, VEC>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)),
                      dim3(256), 0, s, a);
  }
  a.chunks = (a.units + 256 * kItems - 1) / (256 * kItems);
  a.segment = (a.units + a.chunks - 1) / a.chunks;
  const unsigned threads = ((a.segment + kItems - 1) / kItems + 31) / 32 * 32;
  return launch_pdl(k_dropout<T, VEC>, dim3(static_cast<unsigned>((a.rows + kRows - 1) / kRows * a.chunks)), dim3(threads), 0, s,
                    a);
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
    if (dtype == LORA_BF16)
      return vec ? launch_dropout<__nv_bfloat16, true>(a, st) : launch_dropout<__nv_bfloat16, false>(a, st);
    return vec ? launch_dropout<float, true>(a, st) : launch_dropout<float, false>(a, st);
  });
}
