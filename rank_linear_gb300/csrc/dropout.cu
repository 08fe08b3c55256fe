// dropout.cu -- dropout from a counter-based generator (include/lora_dropout.h;
// the Unsloth essay's recipe table names the rate).
//
// y = keep ? x * scale : 0 with the mask made from (seed, offset, row, column)
// by both directions.  An element moves 4 bytes (bf16) or 8, and takes a quarter
// of the generator's ten rounds: 1.73e12 words a second is all that an otherwise
// empty loop of them makes on the 152 SMs (the 32 x 32 -> 64 products bound it),
// and 1.70e12 elements of bf16 a second is what memory moves.  So what is not the
// generator is kept small: a block's rows and addresses are worked out once; in rows of
// many units a block is at one row at a time, so that the row's share of the first two
// rounds is the same in all its threads.
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
  uint32_t groups, inverse;  // k_dropout_shift: groups of segment + 1 threads, a block
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

// Rows of bf16 that do not begin on 16 bytes, where x and y lie alike past them: a
// thread takes 16 aligned bytes of four rows, of a row's eight columns from 8 v - m on
// (m elements lie between the boundary and the row).  It makes the masks of columns
// 8 v .. 8 v + 7, and has what is before them from its neighbour, by shared memory: a bit
// an element, one word for the four rows.  A group's first thread makes masks only.
// ONE: the block is one group (the rows' share of the first two rounds is common).
// Bound by instructions, at 1.0e12 elements a second: element by element 8191 x 14335
// took 184 us, so 116 (8192 x 14336, aligned: 91); 1800000 x 65 272, so 159.
template <bool ONE>
__global__ void __launch_bounds__(256) k_dropout_shift(const __grid_constant__ Args a) {
  __shared__ uint32_t masks[256];
  griddep_wait();
  griddep_launch_dependents();
  const DropNow now = drop_now(a.drop);
  // groups of segment + 1 threads: threadIdx / that, exact below 256
  const uint32_t group = ONE ? 0 : threadIdx.x * a.inverse >> 16, t = threadIdx.x - group * (a.segment + 1);
  const uint32_t chunk = blockIdx.x % a.chunks;
  const int64_t row = (int64_t(blockIdx.x / a.chunks) * (ONE ? 1 : a.groups) + group) * kRows;
  const int v = static_cast<int>(chunk * a.segment + t) - 1;  // -1: of no column
  const int n = (ONE ? t > a.segment : group >= a.groups) || row >= a.rows ? 0 : a.rows - row < kRows ? static_cast<int>(a.rows - row) : kRows;
  const int cols = static_cast<int>(a.cols);
  const uint64_t x = reinterpret_cast<uint64_t>(a.x), y = reinterpret_cast<uint64_t>(a.y);
  const uint64_t last = x + (uint64_t(a.rows - 1) * a.xs + a.cols) * 2;  // behind x
  const bool mine = t > 0;
  const int64_t at = row * a.xs + 8 * v, to = row * a.ys + 8 * v;
  const uint32_t base = static_cast<uint32_t>((x >> 1) + row * a.xs), step = static_cast<uint32_t>(a.xs);
  Raw8<__nv_bfloat16> in[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int m = static_cast<int>((base + r * step) & 7u), c = 8 * v - m;
    if (!mine || r >= n || c >= cols) continue;
    const uint64_t from = x + (at + r * a.xs - m) * 2;
    const auto *p = reinterpret_cast<const __nv_bfloat16 *>(from);
    if (from >= x && from + 16 <= last) {  // (may hold the neighbours' elements)
      in[r].load(p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k % 2 == 0) in[r].u[k / 2] = 0u;
        if (c + k >= 0 && c + k < cols) in[r].load1(k, p + k);
      }
    }
  }
  // word >= T where word + (2^32 - T) carries (T > 0); the last element's bit first
  uint32_t keep = 0;
  const uint32_t less = 0u - a.drop.threshold;
  auto bit = [&](uint32_t word) {
    uint32_t sum;
    asm("add.cc.u32 %0, %2, %3;\n\taddc.u32 %1, %4, %4;" : "=r"(sum), "=r"(keep) : "r"(word), "r"(less), "r"(keep));
  };
#pragma unroll
  for (int r = kRows - 1; r >= 0; --r) {
#pragma unroll
    for (int h = 1; h >= 0; --h) {
      const uint4 w = drop_words(a.drop, now, static_cast<uint32_t>(2 * v + h), row + r);
      bit(w.w), bit(w.z), bit(w.y), bit(w.x);
    }
  }
  masks[threadIdx.x] = keep;
  __syncthreads();
  if (!mine) return;
  const uint32_t before = masks[threadIdx.x - 1];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int m = static_cast<int>((base + r * step) & 7u), c = 8 * v - m;
    if (r >= n || c >= cols) continue;
    uint32_t bits = ((before >> 8 * r & 255u) | (keep >> 8 * r & 255u) << 8) >> (8 - m);
    bits |= bits << 15;  // elements 2 i and 2 i + 1 at bits 2 i and 16 + 2 i
    Raw8<__nv_bfloat16> out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out.set(i, mul2(in[r].pair(i), both(a.drop.scale)));
      out.u[i] &= (bits >> 2 * i & 0x10001u) * 0xffffu;
    }
    auto *p = reinterpret_cast<__nv_bfloat16 *>(y) + (to + r * a.ys - m);
    if (c >= 0 && c + 8 <= cols) {
      out.store(p);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k >= 0 && c + k < cols) out.store1(k, p + k);
    }
  }
}

// (narrower rows leave most threads at a row's ends)
constexpr uint32_t kShiftCols = 32;
bool shifted(const Args &a) {
  return a.drop.threshold > 0 && a.cols >= kShiftCols && a.cols < (1u << 30) &&  // (columns as int)
         a.xs >= 0 && (reinterpret_cast<uint64_t>(a.x) - reinterpret_cast<uint64_t>(a.y)) % 16 == 0 &&
         (a.xs - a.ys) % 8 == 0;
}
cudaError_t launch_shift(Args a, cudaStream_t s) {
  const uint32_t vectors = (a.cols + 7 + 7) / 8;  // of a row, at most
  a.chunks = (vectors + 254) / 255;
  a.segment = (vectors + a.chunks - 1) / a.chunks;
  if (a.chunks > 1 || a.segment > 128) {  // the cut that leaves the fewest threads idle
    auto cost = [&](uint32_t n) { return n * (((vectors + n - 1) / n + 1 + 31) / 32 * 32); };
    for (uint32_t n = a.chunks + 1, i = 0; i < 8; ++i, ++n)
      if (cost(n) < cost(a.chunks)) a.chunks = n;
    a.segment = (vectors + a.chunks - 1) / a.chunks;
  }
  a.groups = 256 / (a.segment + 1);
  // (one group where that leaves few idle threads: 116000 x 1001 took 121 us with two, 116 so)
  const uint32_t whole = (a.segment + 1 + 31) / 32 * 32;
  if (a.chunks > 1 || (whole > 64 && 8 * (a.segment + 1) >= 7 * whole)) a.groups = 1;
  a.inverse = (65536 + a.segment) / (a.segment + 1);
  const unsigned threads = (a.groups * (a.segment + 1) + 31) / 32 * 32;
  const int64_t per = int64_t(kRows) * a.groups;
  return launch_pdl(a.groups == 1 ? k_dropout_shift<true> : k_dropout_shift<false>, dim3(static_cast<unsigned>((a.rows + per - 1) / per * a.chunks)),
                    dim3(threads), 0, s, a);
}

template <class T, bool VEC>
cudaError_t launch_dropout(Args a, cudaStream_t s) {
  if constexpr (sizeof(T) == 2 && !VEC)
    if (shifted(a)) return launch_shift(a, s);
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
